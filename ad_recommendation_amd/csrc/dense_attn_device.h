// Device helpers of the attention kernels: matrix-core products, LDS tiles and the rows of a wave, which
// sequence a workgroup has, and sums that are not finite.
//
// All products run on the matrix cores as 32x32x16 with fp32 sums.  A product's result has a column
// in a lane and 16 of its 32 rows (8 (r / 4) + 4 (lane / 32) + r % 4 for register r) in that lane's
// registers, and a right operand has a column in a lane and eight consecutive k of 16 there.  The
// kernels put what the softmax runs over into rows (keys where a lane has a query, queries where it
// has a key), so that statistics and rescaling stay within a lane and its partner 32 lanes on, and
// the probabilities become the next product's right operand as they are: which row of the sum
// stands at which k is free as long as the left operand agrees, and the left operand comes out of
// LDS by transposing reads, four rows at any address at a time.
#pragma once

#include <type_traits>

#include "dense_device.h"

namespace emb {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();
constexpr int kThreads = 256;

// The two shapes of a workgroup in training.  Four waves have 128 tokens, 32 each, and share LDS tiles
// of 64 rows, two of each so that one barrier a tile is enough.  One wave has 32 tokens and tiles of 32
// rows to itself: no wave waits for another or is left without tokens by a short sequence, and what the
// rows next to each other read twice is in the caches; see one_wave().
template <int WAVES>
struct Group {
  static constexpr int kTokens = 32 * WAVES;
  static constexpr int kThreads = 64 * WAVES;
  static constexpr int kRows = WAVES == 1 ? 32 : 64;  // of an LDS tile
  static constexpr int kBuffers = WAVES == 1 ? 1 : 2;
};

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x16 mma(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// AGAIN, here and below: not 0 in what a kernel computes once more because its sums were not finite.  The compiler
// would keep what both ways have in common (each address) in registers all along and spill; a lane's number that
// comes about in another way is the second way's own.
template <int AGAIN = 0>
__device__ __forceinline__ int lane_id() {
  if (AGAIN) return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 64 * AGAIN)) - 64 * AGAIN;
  return threadIdx.x & 63;
}
template <int AGAIN>
__device__ __forceinline__ int thread_id() {
  if (AGAIN) return (__builtin_amdgcn_readfirstlane(threadIdx.x) & ~63) + lane_id<AGAIN>();
  return threadIdx.x;
}
// The row of a result that register r of this lane holds.
__device__ __forceinline__ int row_of(int r) { return 8 * (r >> 2) + 4 * (lane_id() >> 5) + (r & 3); }

// ---------------------------------------------------------------- work items
struct Seq {
  int64_t begin;  // first token
  int len, tile;  // tokens; which tile of the sequence this workgroup has
  int index;
};
// A: what has the offsets `off` of n_seq sequences of n_tok tokens.
template <typename A>
__device__ __forceinline__ Seq sequence(const A& a, int b, int tile) {
  Seq s;
  s.index = b;
  s.begin = min(max((int64_t)a.off[b], (int64_t)0), a.n_tok);
  const int64_t end = min(max((int64_t)a.off[b + 1], s.begin), a.n_tok);
  s.len = (int)(end - s.begin);
  s.tile = tile;
  return s;
}
// Tile slot s of a ragged batch, where sequence b's tiles start at slot first(begin, b): a function that
// leaves each sequence room for its tiles without a pass over the lengths (begin / tile + b does: the
// tiles of a length l that starts anywhere number at most l / tile + 1).  64 lanes look for the
// sequence together.  Offsets are clamped to the tokens.
template <typename A, typename F>
__device__ __forceinline__ Seq find_tile(const A& a, int slot, F first) {
  auto start = [&](int b) { return first(min(max((int64_t)a.off[b], (int64_t)0), a.n_tok), b); };
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
  Seq s = sequence(a, lo, 0);
  s.tile = (int)max((int64_t)slot - (int64_t)first(s.begin, lo), (int64_t)-1);
  return s;
}

// Sets x[r] to `hidden` where query i does not see key j0 + row_of(r): the distance i - j, taken as an
// unsigned number, is below the window, or below all others for a sink.  Few tiles need it; the empty
// statement keeps the compiler from doing it in all of them and choosing afterwards.
// Returns a bit for each register whose key it sees.
template <int AGAIN>
__device__ __forceinline__ uint32_t hide_keys(const AttnArgs& a, int i, int j0, f32x16& x, float hidden) {
  asm volatile("");
  const int half = lane_id<AGAIN>() >> 5, d = i - j0 - 4 * half, sinks = a.sinks - j0 - 4 * half;
  uint32_t see = 0xFFFF;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int e = 8 * (r >> 2) + (r & 3);
    const uint32_t limit = e < sinks ? 0x7FFFFFFFu : (uint32_t)a.window;
    if ((uint32_t)(d - e) >= limit) {
      x[r] = hidden;
      see &= ~(1u << r);
    }
  }
  return see;
}

// ---------------------------------------------------------------- LDS tiles
// Rows of a head in LDS, read in two ways: 16-byte pieces of 16 rows at once (left operands) and, by the
// transposing reads, four pieces of four consecutive rows at once.  LDS has 64 banks of 4 bytes, so
// both are without conflict if the 16 rows' pieces, and the four rows' four pieces, lie in 16 different
// places of 256 bytes.  (With rows in order and 16 bytes between them the second kind met itself: half
// the cycles that the forward kept LDS busy.)
//
// Through registers: an odd number of pieces a row, row r of each 16 at place 4 (r % 4) + r / 4.
// Zeros past the last row and column.
template <typename T, int DH, int ROWS, int THREADS, int AGAIN = 0>
struct RegisterTile {
  static constexpr int kPieces = DH / 8, kRow = DH * 2 + 16, kBytes = ROWS * kRow;
  static constexpr int kRegs = ROWS * kPieces / THREADS;
  __device__ static __forceinline__ int at(int row, int piece) {
    return ((row & ~15) | (row & 3) << 2 | (row >> 2 & 3)) * kRow + piece * 16;
  }
  struct Reads {  // where a lane reads in a tile
    int l, t;
    __device__ __forceinline__ Reads() {
      const int n = lane_id<AGAIN>();
      l = at(n & 31, n >> 5);
      t = at(4 * (n >> 5) + ((n & 15) >> 2), ((n >> 4) & 1) * 2) + (n & 3) * 8;
    }
    __device__ __forceinline__ int left(int row0, int ks) const { return l + row0 * kRow + ks * 32; }
    __device__ __forceinline__ int left_t(int row0, int db, int half) const {
      return t + (row0 + 2 * half) * kRow + db * 64;  // eight rows on are two places
    }
  };
  u32x4 r[kRegs];
  // Rows row0 .. row0 + ROWS - 1 of a head, which has `end` of them.
  __device__ __forceinline__ void load(char*, const T* base, int64_t stride, int row0, int end, int D) {
#pragma unroll
    for (int n = 0; n < kRegs; ++n) {
      const int idx = thread_id<AGAIN>() + n * THREADS;
      const int row = row0 + idx / kPieces, col = idx % kPieces * 8;
      r[n] = u32x4{0, 0, 0, 0};
      if (row < end && col < D) r[n] = *reinterpret_cast<const u32x4*>(base + row * stride + col);
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int n = 0; n < kRegs; ++n) {
      const int idx = thread_id<AGAIN>() + n * THREADS;
      *reinterpret_cast<u32x4*>(lds + at(idx / kPieces, idx % kPieces)) = r[n];
    }
  }
  __device__ static __forceinline__ void arrived() {}
};

// Straight from memory to LDS, where heads have DH columns: a wave's load fills 1024 bytes in order, so a
// row's pieces are exchanged by its number instead of set apart, by the address that a lane loads from.
// The last row stands for those past it; no query sees them, and no row past `end` is read.  Against
// registers: no moves, no LDS writes, 32 registers fewer; forward of 17.2k tokens, 16 heads of 128,
// window 1024: 193 -> 172 us.
template <typename T, int DH, int ROWS, int THREADS, int AGAIN = 0>
struct DirectTile {
  static constexpr int kPieces = DH / 8, kRow = DH * 2, kBytes = ROWS * kRow;
  static constexpr int kSpan = 16 / kPieces;  // rows in 256 bytes
  static constexpr int kAtOnce = 64 / kPieces;  // rows of a wave's load
  static constexpr int kLoads = ROWS / kAtOnce / (THREADS / 64);
  static_assert(kLoads * kAtOnce * (THREADS / 64) == ROWS, "whole loads");
  __device__ static __forceinline__ int exchange(int row) { return (row & 3) / kSpan << 2 | (row >> 2 & 3); }
  __device__ static __forceinline__ int at(int row, int piece) { return row * kRow + (piece ^ exchange(row)) * 16; }
  struct Reads {
    int l[DH / 16], t[DH / 32][2];
    __device__ __forceinline__ Reads() {
      const int n = lane_id<AGAIN>(), row = n & 31;
#pragma unroll
      for (int ks = 0; ks < DH / 16; ++ks) l[ks] = at(row, 2 * ks + (n >> 5));
#pragma unroll
      for (int db = 0; db < DH / 32; ++db)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = 4 * (n >> 5) + ((n & 15) >> 2) + 8 * half;
          const int piece = db * 4 + ((n >> 4) & 1) * 2 + ((n & 3) >> 1);
          t[db][half] = at(r, piece) + (n & 1) * 8;
        }
    }
    __device__ __forceinline__ int left(int row0, int ks) const { return l[ks] + row0 * kRow; }
    __device__ __forceinline__ int left_t(int row0, int db, int half) const { return t[db][half] + row0 * kRow; }
  };
  // The compiler would wait for every load to LDS that is under way before each transposing read, of
  // whichever buffer; it is told nothing, and arrived() waits.  The load has no register to write.
  __device__ static __forceinline__ void load_piece(const char* p, uint32_t off, char* lds) {
    typedef __attribute__((address_space(3))) char* Lds;
    const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(Lds)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(off), "s"(p)
                 : "memory", "m0");
  }
  __device__ __forceinline__ void load(char* lds, const T* base, int64_t stride, int row0, int end, int) {
    const int wave = __builtin_amdgcn_readfirstlane(thread_id<AGAIN>() >> 6), lane = lane_id<AGAIN>();
    const int from = min(row0, end - 1), last = end - 1 - from;
    const char* p = reinterpret_cast<const char*>(base + from * stride);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int first = (wave + n * (THREADS / 64)) * kAtOnce, row = first + lane / kPieces;
      const int piece = (lane % kPieces) ^ exchange(row);
      // a tile's rows are within 2^31 bytes of one another: see direct()
      const uint32_t off = (uint32_t)(min(row, last) * ((int)stride * 2) + piece * 16);
      load_piece(p, off, lds + first * kRow);
    }
  }
  __device__ __forceinline__ void store(char*) const {}
  // A barrier does not wait for loads to LDS.
  __device__ static __forceinline__ void arrived() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  }
};

template <typename T, int DH, int ROWS, int THREADS, bool DIRECT, int AGAIN = 0>
using TileOf = std::conditional_t<DIRECT, DirectTile<T, DH, ROWS, THREADS, AGAIN>,
                                  RegisterTile<T, DH, ROWS, THREADS, AGAIN>>;

// Left operand: rows row0 .. row0 + 31, columns 16 ks .. 16 ks + 15 as k.
template <typename T, typename R>
__device__ __forceinline__ typename Vec8<T>::t left(const char* lds, const R& r, int row0, int ks) {
  return *reinterpret_cast<const typename Vec8<T>::t*>(lds + r.left(row0, ks));
}
// Left operand, transposed: columns 32 db .. 32 db + 31 as rows, rows row0 .. row0 + 15 as k, in the
// order in which a result's registers hold them.
template <typename T, typename R>
__device__ __forceinline__ typename Vec8<T>::t left_t(const char* lds, const R& r, int row0, int db) {
  typedef __attribute__((address_space(3))) i16x4* Lds;
  const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(lds + r.left_t(row0, db, 0)));
  const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(lds + r.left_t(row0, db, 1)));
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
__device__ __forceinline__ typename Vec8<T>::t right_of(const f32x16& p, int r) {
  const f32x8 x = {p[r], p[r + 1], p[r + 2], p[r + 3], p[r + 4], p[r + 5], p[r + 6], p[r + 7]};
  return __builtin_convertvector(x, typename Vec8<T>::t);
}

// The 32 rows of a wave, to right operands and from results.  A lane has a row of its own there, 16 or
// 8 bytes at a time, which in memory are scattered pieces of 32 rows; so rows pass through the wave's
// part of LDS (`part`, from row `first` of a tile on) and memory sees whole ones.  Backward of 512 short
// histories: writing results piece by piece took 23 of dq's 92 us.
template <typename T, int DH, typename TILE, int AGAIN = 0>
struct WaveRows {
  static constexpr int kPieces = DH / 8, kRegs = 32 * kPieces / 64;
  u32x4 r[kRegs];
  // the first `rows` of the 32 from token tok on; zeros past them and past D columns
  __device__ __forceinline__ void load(const EmbHeads& t, int64_t tok, int head, int rows, int D) {
    const T* p = static_cast<const T*>(t.p) + tok * t.tok + head * t.head;
#pragma unroll
    for (int n = 0; n < kRegs; ++n) {
      const int idx = lane_id<AGAIN>() + n * 64, row = idx / kPieces, col = idx % kPieces * 8;
      r[n] = u32x4{0, 0, 0, 0};
      if (row < rows && col < D) r[n] = *reinterpret_cast<const u32x4*>(p + row * t.tok + col);
    }
  }
  __device__ __forceinline__ void to_right(char* part, int first, const typename TILE::Reads& at,
                                           typename Vec8<T>::t (&f)[DH / 16]) const {
    wave_sync();
#pragma unroll
    for (int n = 0; n < kRegs; ++n) {
      const int idx = lane_id<AGAIN>() + n * 64;
      *reinterpret_cast<u32x4*>(part + TILE::at(first + idx / kPieces, idx % kPieces)) = r[n];
    }
    wave_sync();
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) f[ks] = left<T>(part, at, first, ks);
  }
  // Rows of results that hold them as columns (one per 32 of their elements), but those in `skip`.
  __device__ static __forceinline__ void store(const EmbHeads& t, int64_t tok, int head, int rows, int D,
                                               char* part, int first, const f32x16 (&x)[DH / 32], float by,
                                               uint32_t skip) {
    typedef T V __attribute__((ext_vector_type(4)));
    const int own = lane_id<AGAIN>() & 31, half = lane_id<AGAIN>() >> 5;
    wave_sync();
#pragma unroll
    for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 v = {x[db][4 * g] * by, x[db][4 * g + 1] * by, x[db][4 * g + 2] * by, x[db][4 * g + 3] * by};
        *reinterpret_cast<V*>(part + TILE::at(first + own, db * 4 + g) + half * 8) = __builtin_convertvector(v, V);
      }
    }
    wave_sync();
    T* p = static_cast<T*>(t.p) + tok * t.tok + head * t.head;
#pragma unroll
    for (int n = 0; n < kRegs; ++n) {
      const int idx = lane_id<AGAIN>() + n * 64, row = idx / kPieces, col = idx % kPieces * 8;
      const u32x4 v = *reinterpret_cast<const u32x4*>(part + TILE::at(first + row, idx % kPieces));
      if (row < rows && col < D && !(skip >> row & 1)) *reinterpret_cast<u32x4*>(p + row * t.tok + col) = v;
    }
  }
  // LDS accesses of one wave are carried out in order; this keeps the compiler to that order.
  __device__ static __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
};

// Writes a lane's row from results that hold it as a column (one per 32 of its elements).
template <typename T, int DH, int AGAIN = 0>
__device__ __forceinline__ void store_row(const EmbHeads& t, int64_t tok, int head, int D,
                                          const f32x16 (&x)[DH / 32], float by) {
  typedef T V __attribute__((ext_vector_type(4)));
  T* p = static_cast<T*>(t.p) + tok * t.tok + head * t.head;
#pragma unroll
  for (int db = 0; db < DH / 32; ++db) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = db * 32 + 8 * g + 4 * (lane_id<AGAIN>() >> 5);
      const f32x4 v = {x[db][4 * g] * by, x[db][4 * g + 1] * by, x[db][4 * g + 2] * by, x[db][4 * g + 3] * by};
      if (col < D) *reinterpret_cast<V*>(p + col) = __builtin_convertvector(v, V);
    }
  }
}

// ---------------------------------------------------------------- what is not finite
// A product adds 0 * x for a pair that does not see each other, which is NaN where x is not finite; and in fp16
// the gradient of a score, which is rounded to 16 bits before its product, is infinite past 65504.  So where sums of
// a workgroup come out not finite it computes them once more, still on the matrix cores, from the pairs that
// see each other alone: what is finite with finite_of and fit, and what is not with add_odd.  It costs a look at
// the sums while they are finite.  8614 tokens, 16 and 8 heads of 128, window 1024, bf16, with an infinity in
// each row of dout, or of v: backward 1.30 ms, forward 0.43; 81 and 31 by one wave that goes over a row's pairs.
template <int N>
__device__ __forceinline__ bool not_finite(const f32x16 (&x)[N]) {
  float z[4] = {0.f, 0.f, 0.f, 0.f};  // four chains: a wave waits for each addition
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r & 3] = fmaf(x[n][r], 0.f, z[r & 3]);
  return z[0] + z[1] + (z[2] + z[3]) != 0.f;
}
// Whether any wave of a workgroup says so, and a barrier.
template <int WAVES>
__device__ __forceinline__ bool any_wave(bool b, uint32_t (&said)[WAVES]) {
  const uint32_t mine = __any(b);
  if (WAVES == 1) {
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(mine) != 0;
  }
  if (lane_id() == 0) said[threadIdx.x >> 6] = mine;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) all |= said[w];
  return __builtin_amdgcn_readfirstlane(all) != 0;
}

// Which of a vector's elements are not finite (all ones), and the vector without them.
template <typename T> constexpr short kTop = std::is_same<T, _Float16>::value ? 0x7C00 : 0x7F80;  // an infinity's bits
template <typename T>
__device__ __forceinline__ i16x8 odd_of(typename Vec8<T>::t x) {
  return (__builtin_bit_cast(i16x8, x) & 0x7FFF) >= kTop<T>;
}
template <typename T>
__device__ __forceinline__ typename Vec8<T>::t finite_of(typename Vec8<T>::t x) {
  return __builtin_bit_cast(typename Vec8<T>::t, (i16x8)(__builtin_bit_cast(i16x8, x) & ~odd_of<T>(x)));
}
// Ones where the pairs see each other, for registers r0 to r0 + 7: `see` has a bit for each.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::t ones(uint32_t see, int r0) {
  typename Vec8<T>::t x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (T)(see >> (r0 + i) & 1 ? 1.f : 0.f);
  return x;
}
// To sum += A B, what A's elements that are not finite add.  Of B it takes `one`, 1 for the pairs that see each
// other and 0 for the rest, and `signs`, 0 for a B of zero or of no known sign.  A product of small whole numbers
// gives, for each element of the sum, 256 times how many of its pairs see something not finite, plus the signs of
// what they add: +1 or -1 for an infinity times a number, 0 for what is NaN.
template <typename T>
__device__ __forceinline__ void add_odd(f32x16& sum, typename Vec8<T>::t a, typename Vec8<T>::t one,
                                        typename Vec8<T>::t signs) {
  typedef typename Vec8<T>::t V8;
  constexpr short kOne = std::is_same<T, _Float16>::value ? 0x3C00 : 0x3F80;
  constexpr short kMany = kOne + 8 * (0x8000 - kTop<T>);  // 256
  const i16x8 odd = odd_of<T>(a), x = __builtin_bit_cast(i16x8, a);
  const u32x4 some = __builtin_bit_cast(u32x4, odd);
  if (!__any(some[0] | some[1] | some[2] | some[3])) return;
  f32x16 n = mma(__builtin_bit_cast(V8, (i16x8)(odd & kMany)), one, f32x16{});
  n = mma(__builtin_bit_cast(V8, (i16x8)(((x & 0x7FFF) == kTop<T>) & (kOne | (x & (short)0x8000)))), signs, n);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float count = rintf(n[r] * (1.f / 256.f)), sign = n[r] - 256.f * count;
    if (count > 0.f) sum[r] += fabsf(sign) == count ? copysignf(kInf, sign) : __builtin_nanf("");
  }
}
// Brings gradients of scores into the range of 16 bits: x times 2^-by, and sums of such products that stand at
// 2^-by already.  A lane has a query or a key, whose sums are its own and its partner's, so `by` is of the two;
// it grows with the largest so far, as a running maximum does.  bf16 has the range of fp32.
template <typename T, int N>
__device__ __forceinline__ void fit(f32x16& x, f32x16 (&sums)[N], int& by) {
  if constexpr (std::is_same<T, _Float16>::value) {
    float top = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(x[r]) < kInf ? fabsf(x[r]) : 0.f);
    const int more = max(__builtin_amdgcn_frexp_expf(swap32_max(top)) - 15 - by, 0);
    by += more;
    const float down = ldexpf(1.f, -more);
#pragma unroll
    for (int n = 0; n < N; ++n) sums[n] *= down;
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = ldexpf(x[r], -by);
  }
}
template <int N>
__device__ __forceinline__ void unfit(f32x16 (&sums)[N], int by) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int r = 0; r < 16; ++r) sums[n][r] = ldexpf(sums[n][r], by);
}

}  // namespace emb
