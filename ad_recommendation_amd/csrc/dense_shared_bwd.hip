// Backward of the attention of candidates that share a history (see dense_shared.hip):
//
//   delta_i = out_i . dout_i;  p_ij = exp(s_ij - lse_i);  ds_ij = scale p_ij (dout_i . v_j - delta_i)
//   dq_i = sum_j ds_ij k_j;  dk_j = sum_i ds_ij q_i;  dv_j = sum_i p_ij dout_i
//
// dq by query rows as the forward has them; dk and dv of a history by tiles of its keys, which meet every row
// (token, head of the group) of the request, so sums stay in registers and nothing is added up in memory; those of
// own tokens by tiles of them, or, where every token is a candidate, one element at a time from p and ds of the row
// with itself.
//
// In fp16 a score's gradient past 65504 does not fit the second product, and below 2^-14 loses bits there: of thousands
// of events and a small dout all of them are.  So each query's, or key's, stand at a power of two of their own (Fit), and
// probabilities, for dv, at one for all.
#include <algorithm>
#include <initializer_list>

#include "dense_shared_device.h"

namespace emb {

namespace {

// Where score gradients stand in fp16: at f, a power of two, and so do sums of their products; bf16 has the range of fp32.
// They begin at 2^12, where those of most calls have their largest between 2^-6 and 65504.  What comes past that brings all
// to a largest of 2^8, with room to grow, and the sums after it, as a running maximum does; and so does a first largest
// below 2^-6.  So where fp16 has fewer bits, below 2^-14, a score's gradient is off by 2^-37 or 2^-19 of the largest at most.
// A lane has a query or a key, and f is of the two lanes that share it.  300 short requests' backward, 8 and 4 heads of 128,
// takes 161 us so, and 156 with gradients as they come; 200 of candidates of 3 tokens, 8 heads of 64, 112 and 113.
template <typename T>
struct Fit {
  static constexpr bool kOn = std::is_same<T, _Float16>::value;
  float f;
  bool set = false;  // whether there was one of kLeast or more
  static constexpr float kLeast = 1.f / 64;
  __device__ __forceinline__ explicit Fit(float at) : f(kOn ? at : 1.f) {}
  // x stands at f already
  template <int N>
  __device__ __forceinline__ void look(f32x16& x, f32x16 (&sums)[N]) {
    if constexpr (kOn) {
      float top = 0.f;
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(x[r]));
      top = swap32_max(top);  // both lanes decide by the same
      set |= top >= kLeast;
      if (__builtin_expect(__any(top > 65504.f || (!set && top > 0.f)), 0)) move(x, sums, top);
    }
  }
  template <int N>
  __device__ __forceinline__ void move(f32x16& x, f32x16 (&sums)[N], float top) {
    top = fminf(top, 0x1p127f);  // of what is not finite the sums are not either
    // not past 2^64, so that f times any product of fp16's numbers is finite
    const int most = 65 - __builtin_amdgcn_frexp_expf(f), to = 9 - __builtin_amdgcn_frexp_expf(top);
    const float by = top > 65504.f || (!set && top > 0.f) ? ldexpf(1.f, min(to, most)) : 1.f;
    f *= by;
    set |= top > 0.f;
    x *= by;
#pragma unroll
    for (int n = 0; n < N; ++n) sums[n] *= by;
  }
  // What sums that stand at f, and at 2^raised besides, are multiplied by.
  __device__ __forceinline__ float back(int raised = 0) const {
    return kOn ? ldexpf(1.f, 1 - __builtin_amdgcn_frexp_expf(f) - raised) : 1.f;
  }
};
constexpr int kRaised = 12;
// Probabilities of the products for dv stand there in fp16, so that they have all their bits down to 2^-26.
template <typename T> constexpr int kRaisedP = Fit<T>::kOn ? kRaised : 0;

// ---------------------------------------------------------------- dq
// What a lane's row has throughout: its operands, delta and lse; also writes delta.
template <typename T, int DH>
struct QueryRow {
  typename Vec8<T>::t q[DH / 16], d[DH / 16];
  float delta, lse;
};
template <typename T, int DH>
__device__ __forceinline__ float row_delta(const typename Vec8<T>::t (&out)[DH / 16],
                                           const typename Vec8<T>::t (&d)[DH / 16]) {
  float s = 0.f;
#pragma unroll
  for (int ks = 0; ks < DH / 16; ++ks)
#pragma unroll
    for (int e = 0; e < 8; ++e) s += (float)out[ks][e] * (float)d[ks][e];
  return swap32_sum(s);
}

// A tile of 32 keys at row at0 of LDS tiles: dq += ds k.  OWN: of keys j0 on the row sees lo to hi, and of an `odd`
// tile, whose keys are not all finite, what is not stays out of the second product.  Otherwise the first n are there, and
// seen.
template <typename T, int DH, bool OWN, typename R>
__device__ __forceinline__ void dq_meet(const char* kt, const char* vt, const R& at, int at0, int n, int lo, int hi,
                                        int j0, const QueryRow<T, DH>& w, float c, f32x16 (&dq)[DH / 32], Fit<T>& fit,
                                        bool odd = false) {
  typedef typename Vec8<T>::t V8;
  f32x16 sc = {}, dp = {};
#pragma unroll
  for (int ks = 0; ks < DH / 16; ++ks) {
    sc = mma(left<T>(kt, at, at0, ks), w.q[ks], sc);
    dp = mma(left<T>(vt, at, at0, ks), w.d[ks], dp);
  }
  f32x16 ds;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float x = Fit<T>::kOn ? fmaf(dp[r], fit.f, -w.delta * fit.f) : dp[r] - w.delta;
    ds[r] = __builtin_amdgcn_exp2f(fmaf(sc[r], c, -w.lse)) * x;
  }
  if (OWN) hide_outside<3>(lo, hi, j0, ds, 0.f);
  else if (n < 32) hide_from(n, 0, ds, 0.f);
  fit.look(ds, dq);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const V8 b = right_of<T>(ds, 8 * k);
#pragma unroll
    for (int db = 0; db < DH / 32; ++db) {
      V8 x = left_t<T>(kt, at, at0 + 16 * k, db);
      if (OWN && odd) {
        asm volatile("");  // a branch, and not a choice in every tile
        x = finite_of<T>(x);
      }
      dq[db] = mma(x, b, dq[db]);
    }
  }
}

// The row's own token alone, on the vector unit; p and ds go to a.self for that token's dk and dv.
template <typename T, int DH>
__device__ __forceinline__ void dq_self(const SharedArgs& a, int64_t tok, int kh, int qh, bool live,
                                        const QueryRow<T, DH>& w, float c, f32x16 (&dq)[DH / 32], float f) {
  const T* kp = static_cast<const T*>(a.k.p) + tok * a.k.tok + kh * a.k.head;
  const T* vp = static_cast<const T*>(a.v.p) + tok * a.v.tok + kh * a.v.head;
  asm volatile("" ::: "memory");  // one row after the other: the registers are full
  const float s = dot_row<T, DH>(w.q, kp, live, a.dim);
  asm volatile("" ::: "memory");
  const float dp = dot_row<T, DH>(w.d, vp, live, a.dim);
  if (!live) return;
  const float p = __builtin_amdgcn_exp2f(fmaf(s, c, -w.lse)), ds = p * (dp - w.delta), x = ds * f;
  const int64_t at = (int64_t)qh * a.n_tok + tok;
  if (lane_id<3>() < 32) a.self[at] = p;
  else a.self[(int64_t)a.q_heads * a.n_tok + at] = ds;
  typedef T V __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = db * 32 + 8 * g + 4 * (lane_id<3>() >> 5);
      f32x4 k = {};
      if (col < a.dim) k = __builtin_convertvector(*reinterpret_cast<const V*>(kp + col), f32x4);
#pragma unroll
      for (int e = 0; e < 4; ++e) dq[db][4 * g + e] += x * k[e];
    }
  }
}

// Waves of a SIMD.  Direct tiles and no token met alone leave 64-wide heads registers for four.
template <int DH, bool LEAN>
constexpr int dq_waves = DH == 128 ? 2 : DH == 64 && !LEAN ? 3 : 4;

// 128 rows a workgroup, 32 a wave, tiles of 64 keys in LDS, as in the forward.  8 requests of up to 512 candidates and
// 4095 events, 16 and 8 heads of 128, bf16: 95 us, matrix cores busy 35 % of the time; 200 of up to 120 tokens and 500
// events, 8 heads of 64, fp16: 68 us for 197 MB, each workgroup's loads one after the other.
template <typename T, int DH, bool DIRECT, bool TILES>
__global__ void __launch_bounds__(256, (dq_waves<DH, DIRECT && TILES>)) shared_dq(SharedArgs a, int splits, int unit) {
  typedef TileOf<T, DH, 64, 256, DIRECT> Tile;
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
  const int wave = uniform(threadIdx.x >> 6);
  const int r0 = s.tile * kTile, rw = r0 + wave * 32, h0 = kh * a.group, last = min(r0 + kTile, rows) - 1;

  typedef PackedRows<T, DH, Tile> Rows;
  Rows ql, dl, ol;
  ql.load(a, a.q, s.begin, h0, rw, rows);
  dl.load(a, a.dout, s.begin, h0, rw, rows);
  ol.load(a, a.out, s.begin, h0, rw, rows);
  const HistoryTiles<kRows> tiles(hist);
  const T* hk = history_of<T>(a, a.hk, hist, s.index, kh);
  const T* hv = history_of<T>(a, a.hv, hist, s.index, kh);
  Tile kl, vl;
  auto load = [&](int it, char (*to)[kBytes]) {
    kl.load(to[0], hk, a.hk.tok, tiles.key0(it), tiles.end(it), a.dim);
    vl.load(to[1], hv, a.hv.tok, tiles.key0(it), tiles.end(it), a.dim);
  };
  if (share.first < share.end) load(share.first, lds[0]);
  const typename Tile::Reads at;
  char* const part = lds[1][wave >> 1];  // a wave's own part of the tiles that the first step does not use
  const int part0 = 32 * (wave & 1);
  QueryRow<T, DH> w;
  ql.to_right(part, part0, at, w.q);
  dl.to_right(part, part0, at, w.d);
  {
    typename Vec8<T>::t out[DH / 16];
    ol.to_right(part, part0, at, out);
    w.delta = row_delta<T, DH>(out, w.d);
  }
  const float c = a.scale * kLog2e;
  {
    const int r = rw + (lane_id() & 31);
    const Row row = row_at(a, min(r, last));
    const int64_t stat = (int64_t)(h0 + row.g) * a.n_tok + s.begin + row.tok;
    if (split == 0 && r < rows && lane_id() < 32) a.delta[stat] = w.delta;
    w.lse = r < rows ? a.lse[stat] * kLog2e : kInf;
  }
  f32x16 dq[DH / 32] = {};
  Fit<T> fit(1 << kRaised);  // of dq
  auto meet = [&](int it, char (*now)[kBytes], char (*next)[kBytes]) {
    kl.store(now[0]);
    vl.store(now[1]);
    if (!DIRECT && it + 1 < share.end) load(it + 1, next);
    Tile::arrived();
    __syncthreads();  // this tile is there, and the other buffer is no longer read
    if (DIRECT && it + 1 < share.end) load(it + 1, next);
    if (rw >= rows) return;
    const int n = tiles.end(it) - tiles.key0(it);
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
      if (32 * sub < n)
        dq_meet<T, DH, false>(now[0], now[1], at, 32 * sub, n - 32 * sub, 0, 0, 0, w, c, dq, fit);
  };
  // two tiles a turn, so that the buffers' places are constants
  for (int it = share.first; it < share.end; it += 2) {
    meet(it, lds[0], lds[1]);
    if (it + 1 < share.end) meet(it + 1, lds[1], lds[0]);
  }

  const int r = rw + (lane_id<3>() & 31);
  const bool live = r < rows;
  const Row row = row_at(a, live ? r : last);
  if (split != share.count - 1) {
    // own tokens are met by the last workgroup of a row
  } else if constexpr (!TILES) {
    dq_self<T, DH>(a, s.begin + row.tok, kh, h0 + row.g, live, w, c, dq, fit.f);
  } else {
    typedef RegisterTile<T, DH, kRows, 256, 3> OwnTile;
    const typename OwnTile::Reads own_at;
    const int lo = first_of(a, s, row.tok), end = uniform(row_at(a, last).tok) + 1;
    for (int j0 = uniform(first_of(a, s, row_at(a, r0).tok)); j0 < end; j0 += kRows) {
      __syncthreads();  // the tile before is done with
      bool odd = false;
      {
        OwnTile tile;
        tile.load(nullptr, static_cast<const T*>(a.k.p) + s.begin * a.k.tok + kh * a.k.head, a.k.tok, j0, end, a.dim);
#pragma unroll
        for (int n = 0; n < OwnTile::kRegs; ++n) only_finite<T>(tile.r[n], odd);
        tile.store(lds[0][0]);
        asm volatile("" ::: "memory");  // one after the other: two would not fit the registers
        tile.load(nullptr, static_cast<const T*>(a.v.p) + s.begin * a.v.tok + kh * a.v.head, a.v.tok, j0, end, a.dim);
        tile.store(lds[0][1]);
      }
      odd = any_wave<4>(odd, said);
      if (rw >= rows) continue;
      if (odd)
        add_odd_own<T, DH>(a, a.k, s.begin, kh, j0, min(j0 + kRows, end), lo, live ? row.tok : -1, true, dq);
      for (int sub = 0; sub < 2; ++sub)
        if (j0 + 32 * sub < end)
          dq_meet<T, DH, true>(lds[0][0], lds[0][1], own_at, 32 * sub, 0, lo, row.tok, j0 + 32 * sub, w, c, dq, fit,
                               odd);
    }
  }
  __syncthreads();  // the tiles are done with
  if (rw >= rows) return;
  const float by = fit.back();
  const int64_t tok = s.begin + row.tok;
  if (splits > 1 && split == 0 && live && lane_id<3>() < 32) *part_count(a, splits, tok, h0 + row.g) = share.count;
  if (share.count > 1) {
    const EmbHeads to{part_of(a, split), 0, (int64_t)a.q_heads * a.dim, a.dim};
    if (live) store_row<float, DH, 3>(to, tok, h0 + row.g, a.dim, dq, by);
    return;
  }
  PackedRows<T, DH, Tile, 3>::store(a, a.dq, s.begin, h0, rw, rows, lds[1][wave >> 1], part0, dq, by * a.scale);
}

// 32 rows a workgroup, where a request has few: its four waves take tiles of 32 keys in turn, and their sums meet
// in LDS.  Bound by a wave's chain of loads and products.
template <typename T, int DH, bool TILES>
__global__ void __launch_bounds__(256, 2) shared_dq_few(SharedArgs a, int splits, int unit) {
  typedef RegisterTile<T, DH, 32, 64> Tile;
  constexpr int kWaves = 4, kRegs = Tile::kRegs, kPieces = Tile::kPieces;
  __shared__ __attribute__((aligned(256))) char lds[kWaves][2][Tile::kBytes];
  int block = blockIdx.x;
  const int kh = block % a.kv_heads;
  block /= a.kv_heads;
  const Unit u = find_unit<32, 32>(a, block, splits, unit);
  if (u.none) return;
  const Seq s = u.s;
  const History hist = u.hist;
  const Share share = u.share;
  const int split = u.split, rows = s.len * a.group;
  const int wave = uniform(threadIdx.x >> 6), lane = lane_id();
  const int r0 = s.tile * 32, h0 = kh * a.group, last = min(r0 + 32, rows) - 1;
  const HistoryTiles<32> tiles(hist);
  const T* hk = history_of<T>(a, a.hk, hist, s.index, kh);
  const T* hv = history_of<T>(a, a.hv, hist, s.index, kh);
  u32x4 kr[kRegs], vr[kRegs];
  auto load = [&](int it) {
    const int j0 = tiles.key0(it), end = tiles.end(it);
#pragma unroll
    for (int n = 0; n < kRegs; ++n) {
      const int idx = lane + n * 64, j = j0 + idx / kPieces, cl = idx % kPieces * 8;
      kr[n] = vr[n] = u32x4{0, 0, 0, 0};
      if (j < end && cl < a.dim) {
        kr[n] = *reinterpret_cast<const u32x4*>(hk + j * a.hk.tok + cl);
        vr[n] = *reinterpret_cast<const u32x4*>(hv + j * a.hv.tok + cl);
      }
    }
  };
  const typename Tile::Reads at;
  char* kt = lds[wave][0];
  char* vt = lds[wave][1];
  QueryRow<T, DH> w;
  {
    typedef PackedRows<T, DH, Tile> Rows;
    Rows x, y;
    typename Vec8<T>::t out[DH / 16];
    x.load(a, a.dout, s.begin, h0, r0, rows);
    y.load(a, a.out, s.begin, h0, r0, rows);
    x.to_right(kt, 0, at, w.d);
    y.to_right(kt, 0, at, out);
    w.delta = row_delta<T, DH>(out, w.d);
    x.load(a, a.q, s.begin, h0, r0, rows);
    x.to_right(kt, 0, at, w.q);
    Rows::W::wave_sync();
  }
  int it = share.first + wave;
  if (it < share.end) load(it);
  const float c = a.scale * kLog2e;
  {
    const int r = r0 + (lane & 31);
    const Row row = row_at(a, min(r, last));
    const int64_t stat = (int64_t)(h0 + row.g) * a.n_tok + s.begin + row.tok;
    if (split == 0 && r < rows && threadIdx.x < 32) a.delta[stat] = w.delta;
    w.lse = r < rows ? a.lse[stat] * kLog2e : kInf;
  }
  f32x16 dq[DH / 32] = {};
  Fit<T> fit(1 << kRaised);
  for (; it < share.end; it += kWaves) {
#pragma unroll
    for (int n = 0; n < kRegs; ++n) {
      const int idx = lane + n * 64, to = Tile::at(idx / kPieces, idx % kPieces);
      *reinterpret_cast<u32x4*>(kt + to) = kr[n];
      *reinterpret_cast<u32x4*>(vt + to) = vr[n];
    }
    if (it + kWaves < share.end) load(it + kWaves);
    WaveRows<T, DH, Tile>::wave_sync();
    dq_meet<T, DH, false>(kt, vt, at, 0, tiles.end(it) - tiles.key0(it), 0, 0, 0, w, c, dq, fit);
    WaveRows<T, DH, Tile>::wave_sync();
  }
  const int r = r0 + (lane_id<3>() & 31);
  const bool live = r < rows;
  const Row row = row_at(a, live ? r : last);
  if (split != share.count - 1) {
    // own tokens are met by the last workgroup of a row
  } else if constexpr (!TILES) {
    if (wave == 0) dq_self<T, DH>(a, s.begin + row.tok, kh, h0 + row.g, live, w, c, dq, fit.f);
  } else {
    typedef WaveRows<T, DH, Tile, 3> OwnRows;
    const typename RegisterTile<T, DH, 32, 64, 3>::Reads own_at;
    const int lo = first_of(a, s, row.tok), end = uniform(row_at(a, last).tok) + 1;
    for (int j0 = uniform(first_of(a, s, row_at(a, r0).tok)) + 32 * wave; j0 < end; j0 += 32 * kWaves) {
      OwnRows::wave_sync();
      bool odd = false;
#pragma nounroll
      for (int x = 0; x < 2; ++x) {
        OwnRows rows_;
        rows_.load(x ? a.v : a.k, s.begin + j0, kh, end - j0, a.dim);
#pragma unroll
        for (int n = 0; n < kRegs; ++n) {
          const int idx = lane_id<3>() + n * 64;
          bool its = false;
          only_finite<T>(rows_.r[n], its);
          if (!x) odd |= its;
          *reinterpret_cast<u32x4*>(lds[wave][x] + Tile::at(idx / kPieces, idx % kPieces)) = rows_.r[n];
        }
      }
      OwnRows::wave_sync();
      odd = __any(odd);
      if (odd)
        add_odd_own<T, DH>(a, a.k, s.begin, kh, j0, min(j0 + 32, end), lo, live ? row.tok : -1, true, dq);
      dq_meet<T, DH, true>(kt, vt, own_at, 0, 0, lo, row.tok, j0, w, c, dq, fit, odd);
    }
  }
  const float by = fit.back();
  // the waves meet, as in the forward
  static_assert(sizeof(lds[0]) >= sizeof(float) * 32 * DH, "a wave's sums take its tiles' place");
  f32x4* mine = reinterpret_cast<f32x4*>(lds[wave]);
  WaveRows<T, DH, Tile>::wave_sync();
#pragma unroll
  for (int x = 0; x < DH / 8; ++x) {
    const f32x16 t = dq[x >> 2];
    const int e = (x & 3) * 4;
    mine[x * 64 + lane] = f32x4{t[e] * by, t[e + 1] * by, t[e + 2] * by, t[e + 3] * by};
  }
  __syncthreads();
#pragma unroll
  for (int x = wave; x < DH / 8; x += kWaves) {  // which four rows
    const int d = x * 8 + 4 * (lane >> 5);
    f32x4 t = {};
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      const f32x4 o = reinterpret_cast<const f32x4*>(lds[v])[x * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] += o[e];
    }
    if (!live || d >= a.dim) continue;
    if (share.count > 1) {
      *reinterpret_cast<f32x4*>(part_of(a, split) + ((s.begin + row.tok) * a.q_heads + h0 + row.g) * a.dim + d) = t;
      continue;
    }
    typedef T V __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] *= a.scale;
    *reinterpret_cast<V*>(row_ptr<T>(a.dq, s.begin, h0, row) + d) = __builtin_convertvector(t, V);
  }
  if (splits > 1 && split == 0 && live && threadIdx.x < 32)
    *part_count(a, splits, s.begin + row.tok, h0 + row.g) = share.count;
}

// What is left when the sums are there, in one launch.  dq of rows that several workgroups shared: a thread adds
// four columns of their parts, in order.  And dk and dv of tokens that are candidates of their own, from p and ds of
// their rows with themselves: a thread has eight columns of a token's key/value head and goes over its heads' group.
// Bound by memory's latency: 11 us for 2050 tokens on average, 16 and 8 heads of 128, up to two parts.
template <typename T, bool SELF>
__global__ void __launch_bounds__(256) shared_finish(SharedArgs a, int splits, int join_blocks) {
  typedef typename Vec8<T>::t V8;
  typedef T V4 __attribute__((ext_vector_type(4)));
  if ((int)blockIdx.x < join_blocks) {
    const int pieces = a.dim / 4;
    const int64_t total = a.n_tok * a.q_heads, i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / pieces;
    const int d = (int)(i - row * pieces) * 4;
    if (row >= total) return;
    const int64_t tok = row / a.q_heads;
    const int qh = (int)(row - tok * a.q_heads), count = min(*part_count(a, splits, tok, qh), splits);
    if (count <= 1 || !in_request(a, tok)) return;  // it has its gradient, or is in no request
    f32x4 t = {};
#pragma unroll 4
    for (int x = 0; x < count; ++x) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + (x * total + row) * a.dim + d);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] += v[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] *= a.scale;
    *reinterpret_cast<V4*>(static_cast<T*>(a.dq.p) + tok * a.dq.tok + qh * a.dq.head + d) =
        __builtin_convertvector(t, V4);
    return;
  }
  if (!SELF) return;
  const int pieces = a.dim / 8;
  const int64_t i = (int64_t)(blockIdx.x - join_blocks) * 256 + threadIdx.x, unit = i / pieces;
  const int col = (int)(i - unit * pieces) * 8;
  const int64_t tok = unit / a.kv_heads;
  const int kh = (int)(unit - tok * a.kv_heads);
  if (tok >= a.n_tok || !in_request(a, tok)) return;
  f32x8 dk = {}, dv = {};
  for (int g = 0; g < a.group; ++g) {
    const int h = kh * a.group + g;
    const int64_t at = (int64_t)h * a.n_tok + tok;
    const float p = a.self[at], ds = a.self[(int64_t)a.q_heads * a.n_tok + at];
    const f32x8 q = widen(*reinterpret_cast<const V8*>(static_cast<const T*>(a.q.p) + tok * a.q.tok + h * a.q.head + col));
    const f32x8 d = widen(*reinterpret_cast<const V8*>(static_cast<const T*>(a.dout.p) + tok * a.dout.tok +
                                                       h * a.dout.head + col));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dk[e] = fmaf(ds, q[e], dk[e]);
      dv[e] = fmaf(p, d[e], dv[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) dk[e] *= a.scale;
  *reinterpret_cast<V8*>(static_cast<T*>(a.dk.p) + tok * a.dk.tok + kh * a.dk.head + col) = __builtin_convertvector(dk, V8);
  *reinterpret_cast<V8*>(static_cast<T*>(a.dv.p) + tok * a.dv.tok + kh * a.dv.head + col) = __builtin_convertvector(dv, V8);
}

// ---------------------------------------------------------------- dk, dv
// A workgroup has 128 keys of a history for a key/value head and meets the request's rows, 64 a step.  Heads of 64 and
// less: four waves of 32 keys, which hold them as right operands in registers (three waves a SIMD would spill them: 99 us
// instead of 80).  Heads of 128: eight waves, two to each 32 keys with half of a step's rows, and keys and values in LDS.
// The sizes of shared_dq: 137 us, matrix cores busy 31 % of the time, LDS 34 %, waves waiting 44 %; and 105 us for 360
// MB, one or two steps a workgroup, so that finding its request, loads and stores are most of its time.

// 64 rows (token, head of the group) to LDS.
template <typename T, int DH, int THREADS, bool DIRECT>
struct RowsTile : TileOf<T, DH, 64, THREADS, DIRECT> {
  typedef TileOf<T, DH, 64, THREADS, DIRECT> B;
  __device__ __forceinline__ void load(char* lds, const SharedArgs& a, const EmbHeads& t, int64_t begin, int h0, int r0,
                                       int rows) {
    if constexpr (DIRECT) {
      const int wave = uniform(threadIdx.x >> 6), lane = lane_id();
      const int from = min(r0, rows - 1), t0 = uniform(row_at(a, from).tok);
      const char* p = reinterpret_cast<const char*>(static_cast<const T*>(t.p) + (begin + t0) * t.tok + h0 * t.head);
#pragma unroll
      for (int n = 0; n < B::kLoads; ++n) {
        const int first = (wave + n * (THREADS / 64)) * B::kAtOnce, row = first + lane / B::kPieces;
        const int piece = (lane % B::kPieces) ^ B::exchange(row);
        const Row x = row_at(a, min(r0 + row, rows - 1));
        const uint32_t off = (uint32_t)((x.tok - t0) * ((int)t.tok * 2) + x.g * ((int)t.head * 2) + piece * 16);
        B::load_piece(p, off, lds + first * B::kRow);
      }
    } else {
#pragma unroll
      for (int n = 0; n < B::kRegs; ++n) {
        const int idx = threadIdx.x + n * THREADS, row = r0 + idx / B::kPieces, col = idx % B::kPieces * 8;
        B::r[n] = u32x4{0, 0, 0, 0};
        if (row < rows && col < a.dim)
          B::r[n] = *reinterpret_cast<const u32x4*>(row_ptr<const T>(t, begin, h0, row_at(a, row)) + col);
      }
    }
  }
};

template <typename T, int DH, bool DIRECT>
struct DkvTiles {
  static constexpr bool kWide = DH == 128;
  static constexpr int kWaves = kWide ? 8 : 4, kThreads = 64 * kWaves, kShare = kWide ? 2 : 1;
  typedef TileOf<T, DH, 64, kThreads, DIRECT> Tile;
  static constexpr int kBytes = Tile::kBytes;
  char q[2][kBytes], d[2][kBytes];
  char k[kWide ? 2 : 0][kBytes], v[kWide ? 2 : 0][kBytes];
  float lse[2][64], delta[2][64];
  __device__ __forceinline__ char* part(int wave) {
    if (kWide) return wave & 2 ? v[0] : k[0];
    return (wave & 2 ? d : q)[1];
  }
};

// Adds the sums of the upper half of eight waves to those of the lower half, through LDS; each times its `by`.
template <int N>
__device__ __forceinline__ void fold_waves(f32x16 (&x)[N], float* lds, int wave, float by) {
  __syncthreads();
  if (wave >= 4) {
#pragma unroll
    for (int k = 0; k < N * 16; ++k) lds[((wave - 4) * N * 16 + k) * 64 + lane_id()] = x[k >> 4][k & 15] * by;
  }
  __syncthreads();
  if (wave < 4) {
#pragma unroll
    for (int k = 0; k < N * 16; ++k) x[k >> 4][k & 15] = fmaf(x[k >> 4][k & 15], by, lds[(wave * N * 16 + k) * 64 + lane_id()]);
  }
}

// Of keys j0 to j1 - 1 of a history: all rows of the request.
template <typename T, int DH, bool DIRECT>
__device__ __forceinline__ void dkv(const SharedArgs& a, DkvTiles<T, DH, DIRECT>& sh, const Seq& s, const History& hist,
                                    int kh, int j0, int j1) {
  typedef typename Vec8<T>::t V8;
  typedef DkvTiles<T, DH, DIRECT> P;
  typedef typename P::Tile Tile;
  constexpr int kRows = 64;
  const int wave = uniform(threadIdx.x >> 6), h0 = kh * a.group;
  const int jrow = 32 * (wave & 3), jw = j0 + jrow, j = jw + (lane_id() & 31);
  const int rows = s.len * a.group;

  RowsTile<T, DH, P::kThreads, DIRECT> ql, dl;
  float stat = 0.f;  // the first 64 threads: lse of a row; as many after them: its delta
  auto load = [&](int b, int r0) {
    ql.load(sh.q[b], a, a.q, s.begin, h0, r0, rows);
    dl.load(sh.d[b], a, a.dout, s.begin, h0, r0, rows);
    if (threadIdx.x < 2 * kRows) {
      const int r = r0 + (threadIdx.x & (kRows - 1));
      const float* p = threadIdx.x < kRows ? a.lse : a.delta;
      // a row that is not there gets probabilities of zero
      stat = threadIdx.x < kRows ? kInf : 0.f;
      if (r < rows) {
        const Row x = row_at(a, r);
        stat = p[(int64_t)(h0 + x.g) * a.n_tok + s.begin + x.tok];
      }
    }
  };
  if (rows > 0) load(0, 0);
  const typename Tile::Reads at;
  typedef WaveRows<T, DH, Tile> Rows;
  V8 k[P::kWide ? 1 : DH / 16], v[P::kWide ? 1 : DH / 16];
  if constexpr (P::kWide) {
    const T* kp = history_of<T>(a, a.hk, hist, 0, kh);
    const T* vp = history_of<T>(a, a.hv, hist, 0, kh);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      Tile kl, vl;
      kl.load(sh.k[x], kp, a.hk.tok, j0 + kRows * x, j1, a.dim);
      vl.load(sh.v[x], vp, a.hv.tok, j0 + kRows * x, j1, a.dim);
      kl.store(sh.k[x]);
      vl.store(sh.v[x]);
    }
  } else {
    // through the buffers that the first step does not use
    Rows kl, vl;
    kl.load(a.hk, hist.row + jw, kh, j1 - jw, a.dim);
    vl.load(a.hv, hist.row + jw, kh, j1 - jw, a.dim);
    kl.to_right(sh.part(wave), 32 * (wave & 1), at, k);
    vl.to_right(sh.part(wave), 32 * (wave & 1), at, v);
  }
  const float c = a.scale * kLog2e;
  f32x16 dk[DH / 32] = {}, dv[DH / 32] = {};
  Fit<T> fit(1.f);  // of dk, beside the probabilities'
  for (int r0 = 0, b = 0; r0 < rows; r0 += kRows, b ^= 1) {
    ql.store(sh.q[b]);
    dl.store(sh.d[b]);
    if (threadIdx.x < kRows) sh.lse[b][threadIdx.x] = stat * kLog2e - kRaisedP<T>;
    else if (threadIdx.x < 2 * kRows) sh.delta[b][threadIdx.x - kRows] = stat;
    if (!DIRECT && r0 + kRows < rows) load(b ^ 1, r0 + kRows);
    Tile::arrived();
    __syncthreads();  // this step's rows are there, and the other buffer is no longer read
    if (DIRECT && r0 + kRows < rows) load(b ^ 1, r0 + kRows);
    if (jw >= j1) continue;
#pragma unroll
    for (int sub_ = 0; sub_ < 2 / P::kShare; ++sub_) {
      const int sub = P::kShare == 2 ? wave >> 2 : sub_;
      if (r0 + 32 * sub >= rows) continue;
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
        const int i = 32 * sub + 8 * g + 4 * (lane_id() >> 5);
        const f32x4 lse = *reinterpret_cast<const f32x4*>(&sh.lse[b][i]);
        const f32x4 delta = *reinterpret_cast<const f32x4*>(&sh.delta[b][i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[4 * g + e] = __builtin_amdgcn_exp2f(fmaf(sc[4 * g + e], c, -lse[e]));
          ds[4 * g + e] = p[4 * g + e] * (dp[4 * g + e] - delta[e]) * (Fit<T>::kOn ? fit.f : 1.f);
        }
      }
      fit.look(ds, dk);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const V8 pb = right_of<T>(p, 8 * x), dsb = right_of<T>(ds, 8 * x);
#pragma unroll
        for (int db = 0; db < DH / 32; ++db) {
          dv[db] = mma(left_t<T>(sh.d[b], at, 32 * sub + 16 * x, db), pb, dv[db]);
          dk[db] = mma(left_t<T>(sh.q[b], at, 32 * sub + 16 * x, db), dsb, dk[db]);
        }
      }
    }
  }
  float by = fit.back(kRaisedP<T>);
  Tile::arrived();  // of keys that no row met
  if (P::kWide) {
    float* fold = reinterpret_cast<float*>(sh.q);
    static_assert(!P::kWide || sizeof(sh.q) + sizeof(sh.d) >= sizeof(float) * 4 * 32 * DH, "room to fold");
    fold_waves(dk, fold, wave, by);
    fold_waves(dv, fold, wave, 1.f);
    by = 1.f;
  } else {
    __syncthreads();  // the tiles are done with
  }
  if (wave >= 4) return;
  // what no row sees gets zeros
  if (rows == 0 || (j < hist.first && j >= hist.sinks)) {
#pragma unroll
    for (int db = 0; db < DH / 32; ++db) dk[db] = dv[db] = f32x16{};
  }
  Rows::store(a.dhk, hist.row + jw, kh, j1 - jw, a.dim, sh.part(wave), 32 * (wave & 1), dk, by * a.scale, 0);
  Rows::store(a.dhv, hist.row + jw, kh, j1 - jw, a.dim, sh.part(wave), 32 * (wave & 1), dv, 1.f / (1 << kRaisedP<T>), 0);
}

struct HistoryBatch {  // of find_tile
  const int32_t* off;
  int64_t n_tok;
  int32_t n_seq;
};

// Waves of a SIMD.
template <int DH>
constexpr int dkv_waves = DH == 32 ? 3 : 2;

// dk and dv of own tokens, where candidates have more than one: a wave has 32 of them for a key/value head and
// meets the rows from there to the end of the last one's candidate, 32 a step.  Candidates are short, and so is this; a
// workgroup of four waves, 128 tokens and 64 rows a step took 90 us where this takes 30 (200 requests of up to 120
// tokens, candidates of 3, 8 heads of 64).
template <typename T, int DH>
struct OwnTiles {
  char tile[2][RegisterTile<T, DH, 32, 64>::kBytes];
  float lse[32], delta[32];
  int first[32], tok[32];
};
template <typename T, int DH>
__device__ __forceinline__ void dkv_own(const SharedArgs& a, OwnTiles<T, DH>& sh, int kh, int slot) {
  typedef typename Vec8<T>::t V8;
  typedef RegisterTile<T, DH, 32, 64> Tile;
  typedef PackedRows<T, DH, Tile> Rows;
  constexpr int kTokens = 32;
  char(&lds)[2][Tile::kBytes] = sh.tile;
  float *const lses = sh.lse, *const deltas = sh.delta;
  int *const firsts = sh.first, *const toks = sh.tok;
  const int h0 = kh * a.group, lane = lane_id();
  const Seq s = uniform(find_tile(a, slot, [](int64_t t, int b) { return t / kTokens + b; }));
  if (s.tile < 0 || (int64_t)s.tile * kTokens >= s.len) return;
  const int j0 = s.tile * kTokens, j1 = min(j0 + kTokens, s.len), j = j0 + (lane & 31), rows = s.len * a.group;
  const typename Tile::Reads at;
  Rows ql, dl;
  float lse = kInf, delta = 0.f;
  int tok = -1, first = 0;
  auto load = [&](int r0) {
    ql.load(a, a.q, s.begin, h0, r0, rows);
    dl.load(a, a.dout, s.begin, h0, r0, rows);
    const int r = r0 + (lane & 31);
    // a row that is not there sees no token
    lse = kInf;
    delta = 0.f;
    tok = -1;
    first = INT32_MAX;
    if (r < rows) {
      const Row x = row_at(a, r);
      const int64_t stat = (int64_t)(h0 + x.g) * a.n_tok + s.begin + x.tok;
      lse = a.lse[stat] * kLog2e - kRaisedP<T>;
      delta = a.delta[stat];
      tok = x.tok;
      first = first_of(a, s, x.tok);
    }
  };
  V8 k[DH / 16], v[DH / 16];
  {
    WaveRows<T, DH, Tile> kl;
    kl.load(a.k, s.begin + j0, kh, j1 - j0, a.dim);
    kl.to_right(lds[0], 0, at, k);
    kl.load(a.v, s.begin + j0, kh, j1 - j0, a.dim);
    kl.to_right(lds[1], 0, at, v);
  }
  const float c = a.scale * kLog2e;
  f32x16 dk[DH / 32] = {}, dv[DH / 32] = {};
  Fit<T> fit(1.f);
  // the next step's rows are not loaded ahead: most have one or two, and there is no register over
  for (int r0 = j0 * a.group; r0 < rows; r0 += 32) {
    load(r0);
    if (uniform(first) >= j1) break;  // candidates from here on begin after the last key
    bool odd = false;
    Rows::W::wave_sync();
#pragma unroll
    for (int n = 0; n < Rows::W::kRegs; ++n) {
      const int idx = lane + n * 64, to = Tile::at(idx / Tile::kPieces, idx % Tile::kPieces);
      *reinterpret_cast<u32x4*>(lds[0] + to) = only_finite<T>(ql.r[n], odd);
      *reinterpret_cast<u32x4*>(lds[1] + to) = only_finite<T>(dl.r[n], odd);
    }
    if (lane < 32) {
      lses[lane] = lse;
      deltas[lane] = delta;
      firsts[lane] = first;
      toks[lane] = tok;
    }
    const bool any_odd = __any(odd);
    Rows::W::wave_sync();
    if (any_odd) {
      for (int i = 0; i < min(32, rows - r0); ++i) {
        const Row x = row_at(a, r0 + i);
        const bool see = j >= firsts[i] && j <= toks[i];
        add_odd_row<T, DH>(row_ptr<const T>(a.q, s.begin, h0, x), a.dim, see, true, dk);
        add_odd_row<T, DH>(row_ptr<const T>(a.dout, s.begin, h0, x), a.dim, see, false, dv);
      }
    }
    f32x16 sc = {}, dp = {};
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) {
      sc = mma(left<T>(lds[0], at, 0, ks), k[ks], sc);
      dp = mma(left<T>(lds[1], at, 0, ks), v[ks], dp);
    }
    f32x16 p, ds;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int i = 8 * g + 4 * (lane >> 5);
      typedef int i32x4 __attribute__((ext_vector_type(4)));
      const f32x4 l4 = *reinterpret_cast<const f32x4*>(&lses[i]), d4 = *reinterpret_cast<const f32x4*>(&deltas[i]);
      const i32x4 f4 = *reinterpret_cast<const i32x4*>(&firsts[i]), t4 = *reinterpret_cast<const i32x4*>(&toks[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __builtin_amdgcn_exp2f(fmaf(sc[4 * g + e], c, -l4[e]));
        const bool seen = j >= f4[e] && j <= t4[e];
        p[4 * g + e] = seen ? x : 0.f;
        ds[4 * g + e] = seen ? x * (dp[4 * g + e] - d4[e]) * (Fit<T>::kOn ? fit.f : 1.f) : 0.f;
      }
    }
    fit.look(ds, dk);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const V8 pb = right_of<T>(p, 8 * x), dsb = right_of<T>(ds, 8 * x);
#pragma unroll
      for (int db = 0; db < DH / 32; ++db) {
        dv[db] = mma(left_t<T>(lds[1], at, 16 * x, db), pb, dv[db]);
        dk[db] = mma(left_t<T>(lds[0], at, 16 * x, db), dsb, dk[db]);
      }
    }
  }
  Rows::W::store(a.dk, s.begin + j0, kh, j1 - j0, a.dim, lds[0], 0, dk, fit.back(kRaisedP<T>) * a.scale, 0);
  Rows::W::store(a.dv, s.begin + j0, kh, j1 - j0, a.dim, lds[1], 0, dv, 1.f / (1 << kRaisedP<T>), 0);
}

// TILES: the first own_blocks workgroups have own tokens, each wave 32 of its own; one launch, so that those, which
// wait for memory most of the time, run beside the histories.
template <typename T, int DH, bool DIRECT, bool TILES>
__global__ void __launch_bounds__((DkvTiles<T, DH, DIRECT>::kThreads), (dkv_waves<DH>))
    shared_dkv(SharedArgs a, int own_blocks) {
  typedef DkvTiles<T, DH, DIRECT> P;
  constexpr int kOwn = TILES ? sizeof(OwnTiles<T, DH>) * P::kWaves : 0;
  __shared__ __attribute__((aligned(1024))) char lds[kOwn > (int)sizeof(P) ? kOwn : sizeof(P)];
  constexpr int kTokens = 128;
  const int kv_heads = a.kv_heads;
  if (TILES && (int)blockIdx.x < own_blocks) {
    const int wave = uniform(threadIdx.x >> 6), unit = blockIdx.x * P::kWaves + wave;
    dkv_own<T, DH>(a, reinterpret_cast<OwnTiles<T, DH>*>(lds)[wave], unit % kv_heads, unit / kv_heads);
    return;
  }
  P& sh = *reinterpret_cast<P*>(lds);
  const int block = blockIdx.x - own_blocks, kh = block % kv_heads, slot = block / kv_heads;
  Seq s;
  History hist;
  int tile;
  if (a.n_seq <= kSorted) {  // as find_unit: those with the most rows first
    const int b = min(lane_id(), a.n_seq - 1);
    const int begin = (int)min(max((int64_t)a.off[b], (int64_t)0), a.n_tok);
    const int len = (int)(min(max((int64_t)a.off[b + 1], (int64_t)begin), a.n_tok) - begin);
    int row, n;
    history_place(a, b, row, n);
    const int units = (n + kTokens - 1) / kTokens;
    const int x = sorted_place(a.n_seq, slot, units, order_of(a.n_seq, units, len), tile);
    if (x < 0) return;
    s.index = x;
    s.begin = __builtin_amdgcn_readlane(begin, x);
    s.len = __builtin_amdgcn_readlane(len, x);
    hist = history_of(a, __builtin_amdgcn_readlane(row, x), __builtin_amdgcn_readlane(n, x));
  } else {
    const Seq h = uniform(find_tile(HistoryBatch{a.hist, a.n_hist, a.n_seq}, slot,
                                    [](int64_t t, int b) { return t / kTokens + b; }));
    if (h.tile < 0 || (int64_t)h.tile * kTokens >= h.len) return;
    hist = history(a, h.index);
    s = uniform(sequence(a, h.index, 0));
    tile = h.tile;
  }
  const int j0 = tile * kTokens;
  // a tile that no row sees has none
  if (j0 >= hist.sinks && j0 + kTokens <= hist.first) s.len = 0;
  dkv<T, DH, DIRECT>(a, sh, s, hist, kh, j0, min(j0 + kTokens, hist.n));
}

// ---------------------------------------------------------------- launches
// Whether tiles may be loaded straight to LDS: whole rows of the kernel's width, and a tile's rows
// within 2^31 bytes of one another.
bool direct(const SharedArgs& a, int width, std::initializer_list<const EmbHeads*> heads) {
  for (const EmbHeads* h : heads) {
    if (h->tok < 0 || h->tok > ((int64_t)1 << 22) || h->head < 0 || h->head * (int64_t)a.group > ((int64_t)1 << 28))
      return false;
  }
  return a.dim == width;
}
int64_t dq_slots(const SharedArgs& a, const SharedBwdPlan& p) { return a.n_tok * a.group / p.rows + a.n_seq; }
int64_t hist_slots(const SharedArgs& a) { return a.n_hist > 0 ? a.n_hist / 128 + a.n_seq : 0; }
int64_t own_blocks(const SharedArgs& a, int waves) {
  return a.n_tok > 0 ? ((a.n_tok / 32 + a.n_seq) * a.kv_heads + waves - 1) / waves : 0;
}
int64_t join_blocks(const SharedArgs& a, const SharedBwdPlan& p) {
  return p.splits > 1 ? (a.n_tok * a.q_heads * (a.dim / 4) + 255) / 256 : 0;
}
int64_t self_blocks(const SharedArgs& a) {
  return a.own == kOwnSelf ? (a.n_tok * a.kv_heads * (a.dim / 8) + 255) / 256 : 0;
}

template <typename T, int DH, bool DIRECT, bool TILES>
hipError_t go(const SharedArgs& a, const SharedBwdPlan& p, hipStream_t st) {
  // a launch that fails is the last one: what comes after it would read what it did not write
  hipError_t e = hipSuccess;
  if (a.n_tok > 0) {
    const dim3 grid((unsigned)(dq_slots(a, p) * a.kv_heads * p.splits));
    if (p.rows == 32) hipLaunchKernelGGL((shared_dq_few<T, DH, TILES>), grid, dim3(256), 0, st, a, p.splits, p.unit);
    else hipLaunchKernelGGL((shared_dq<T, DH, DIRECT, TILES>), grid, dim3(256), 0, st, a, p.splits, p.unit);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  constexpr int kWaves = DkvTiles<T, DH, DIRECT>::kWaves;
  const int64_t own = TILES ? own_blocks(a, kWaves) : 0, dkv = own + hist_slots(a) * a.kv_heads;
  if (dkv > 0) {
    hipLaunchKernelGGL((shared_dkv<T, DH, DIRECT, TILES>), dim3((unsigned)dkv), dim3(64 * kWaves), 0, st, a, (int)own);
    e = hipGetLastError();
  }
  if (e != hipSuccess || a.n_tok == 0) return e;
  const int64_t join = join_blocks(a, p), self = self_blocks(a);
  if (e == hipSuccess && join + self > 0) {
    hipLaunchKernelGGL((shared_finish<T, !TILES>), dim3((unsigned)(join + self)), dim3(256), 0, st, a, p.splits,
                       (int)join);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

SharedBwdPlan plan_shared_bwd(const EmbAttn& a, int64_t n_seq, int64_t n_tok, int64_t n_hist) {
  SharedBwdPlan p{};
  const int64_t group = a.q_heads / a.kv_heads, seen = (int64_t)a.window + a.sinks;
  n_seq = std::max<int64_t>(n_seq, 1);
  const int64_t mean = (n_hist + n_seq - 1) / n_seq, most = std::min(4 * mean, n_hist);
  const auto slots = [&](int64_t rows) {
    return std::max<int64_t>(std::max(n_tok * group / rows, n_seq) * a.kv_heads, 1);
  };
  p.rows = by_32_rows(n_tok * group, n_seq, slots(32), mean) ? 32 : 128;
  const int64_t base = slots(p.rows), least = p.rows == 128 && base >= 128 ? 16 : 8;
  const int tile = p.rows == 32 ? 32 : 64;
  SharedPlan whole{p.rows, 4, 1, 1, 0}, with = whole;
  share_out(whole, base, (mean + tile - 1) / tile, (most + tile - 1) / tile, 400, least);
  share_out(with, base, (std::min(mean, seen) + tile - 1) / tile, (std::min(most, seen) + tile - 1) / tile, 400, least);
  p.splits = std::min(whole.splits, with.splits);  // what is enough without a window is enough with one
  p.unit = with.unit;
  const size_t rows = (size_t)n_tok * a.q_heads;
  const auto room = [](size_t bytes) { return (bytes + 255) & ~(size_t)255; };
  p.off_self = room(rows * sizeof(float));
  p.off_part = p.off_self + room(2 * rows * sizeof(float));
  p.bytes = p.off_part;
  if (p.splits > 1) p.bytes += rows * (p.splits * (size_t)(a.dim + 2) + 1) * sizeof(float);
  return p;
}

int64_t shared_bwd_threads(const SharedArgs& a, const SharedBwdPlan& p) {
  const int waves = a.dim <= 64 ? 4 : 8;
  const int64_t own = a.own == kOwnTiles ? own_blocks(a, waves) : 0;
  return std::max({dq_slots(a, p) * a.kv_heads * p.splits * 256, (own + hist_slots(a) * a.kv_heads) * 64 * waves,
                   (join_blocks(a, p) + self_blocks(a)) * 256});
}

hipError_t launch_shared_bwd(const SharedArgs& a, const SharedBwdPlan& p, hipStream_t st) {
  auto by_width = [&](auto t) {
    typedef decltype(t) T;
    auto by_tiles = [&](auto d) {
      constexpr int DH = decltype(d)::value;
      const bool straight = direct(a, DH, {&a.q, &a.k, &a.v, &a.dout, &a.hk, &a.hv});
      if (a.own == kOwnTiles) return straight ? go<T, DH, true, true>(a, p, st) : go<T, DH, false, true>(a, p, st);
      return straight ? go<T, DH, true, false>(a, p, st) : go<T, DH, false, false>(a, p, st);
    };
    return a.dim <= 32   ? by_tiles(std::integral_constant<int, 32>{})
           : a.dim <= 64 ? by_tiles(std::integral_constant<int, 64>{})
                         : by_tiles(std::integral_constant<int, 128>{});
  };
  return a.dtype == EMB_F16 ? by_width(_Float16{}) : by_width(__bf16{});
}

}  // namespace emb
