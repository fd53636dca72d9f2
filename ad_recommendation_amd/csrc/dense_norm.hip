// The norm after a block, its gate, the scaled residual and the norm before the next block, forward
// and backward.  With inv(z) = rsqrt(mean(z^2) + eps) of a row z:
//   forward   n = w_post * y * inv(y);  r = alpha * x + gate * n;  h = w_pre * r * inv(r)
//   backward  u = dh * w_pre
//             dR = dr + inv(r) * (u - r * inv(r)^2 * mean(u * r))
//             z = gate * dR * w_post;  dx = alpha * dR
//             dy = inv(y) * (z - y * inv(y)^2 * mean(z * y))
//             dgate = dR * n;  dw_post = sum over rows of gate * dR * y * inv(y)
//             dw_pre = sum over rows of dh * r * inv(r)
// Both are bound by HBM: every row is read once into registers, its sums are taken there, and its
// results leave from there.
//
// The backward needs mean(z * y), where z holds dR and so the row's other means.  dR is linear in
// them, so with a = gate * w_post * y
//   sum(z * y) = sum(a * dr) + inv(r) * (sum(a * u) - inv(r)^2 * mean(u * r) * sum(a * r))
// and one exchange of six sums per row is enough, where two exchanges would stand one after the
// other between a row's loads and its stores.
#include "dense_device.h"

namespace emb {

namespace {

constexpr int kThreads = 256;

// Sums K values over the row's TPR threads; every thread gets them.  Rows of at most a wave stay on
// the vector unit; a row of the whole block meets in LDS, in one of two buffers in turn so that one
// barrier a row is enough.
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&s)[K], float (*lds)[kThreads / 64][K], int turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) s[k] = lanes_sum<(TPR < 64 ? TPR : 64)>(s[k]);
  if (TPR > 64) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) lds[turn][w][k] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float t = lds[turn][0][k];
#pragma unroll
      for (int i = 1; i < kThreads / 64; ++i) t += lds[turn][i][k];
      s[k] = t;
    }
  }
}

// Columns of a vector: 16 bytes of the rows' type, so that neighbouring threads read neighbouring 16 bytes.
template <typename T> constexpr int kVec = 16 / sizeof(T);

template <typename T>
__device__ __forceinline__ Vec<float, kVec<T>> wide(Vec<T, kVec<T>> v) {
  return __builtin_convertvector(v, Vec<float, kVec<T>>);
}

// Which columns a thread has: vector c of kVec at col[c].  The last vector of a row whose width is no multiple
// of kVec ends where the row does, so that it is a whole one: its first `twice[c]` columns are the thread
// before's as well.  Both compute them, from the same sums, and write the same bits; sums over the row leave
// them out.  Element by element the end of a row costs seven loads and stores of every wave: 24M
// elements in rows of 500, fp16, forward / backward 50 / 122 us, this way 41 / 60.
// Rows shorter than a vector are read by elements.
template <int W, int TPR, int NC>
struct Columns {
  int col[NC], twice[NC];
  bool some[NC];  // whether there are any
  int width;      // of a vector, the same for all threads
  __device__ __forceinline__ Columns(int D, int lane) {
    width = min(D, W);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * TPR + lane) * W;
      some[c] = at < D;
      col[c] = min(at, D - width);
      twice[c] = at - col[c];
    }
  }
};
// The sum of the squares of the columns that are this thread's alone.
template <int W>
__device__ __forceinline__ float squares(Vec<float, W> x, int twice) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (i >= W - 1 || i >= twice) s += x[i] * x[i];
  return s;
}

// TPR threads take a row, each NC vectors of kVec columns.  32768 x 2048 in bf16, a block a row: 93 us,
// 5.8 TB/s; 100 x 256 in fp16, eight rows a block: 3.2 us.
template <typename T, int TPR, int NC, bool ONCE>
__global__ void __launch_bounds__(kThreads) norm_fwd(NormArgs a) {
  __shared__ float lds[2][kThreads / 64][1];
  constexpr int kRows = kThreads / TPR, W = kVec<T>;
  typedef Vec<T, W> V;
  typedef Vec<float, W> F;
  const int lane = threadIdx.x % TPR;
  const int D = a.dim;
  const T* x = static_cast<const T*>(a.x);
  const T* y = static_cast<const T*>(a.y);
  const T* gate = static_cast<const T*>(a.gate);
  T* r = static_cast<T*>(a.r);
  T* h = static_cast<T*>(a.h);
  const float inv_d = 1.f / (float)D;

  // what all rows share: the weights after the block times a gate vector, the weights before
  const Columns<W, TPR, NC> cl(D, lane);
  F wg[NC], wp[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    wg[c] = F(1.f);
    wp[c] = wg[c];
    if (cl.some[c]) {
      if (a.w_post) wg[c] = load_vec<W>(a.w_post + cl.col[c], cl.width);
      if (a.gate_kind == EMB_GATE_VECTOR) wg[c] *= wide<T>(load_vec<W>(gate + cl.col[c], cl.width));
      if (a.w_pre) wp[c] = load_vec<W>(a.w_pre + cl.col[c], cl.width);
    }
  }
  const int64_t stride = (int64_t)gridDim.x * kRows;
  // the same number of turns for every thread of a block: there are barriers inside
  const int64_t first = (int64_t)blockIdx.x * kRows;
  int turn = 0;
  for (int64_t base = first; base < a.rows; base += stride) {
    const int64_t row = base + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const int64_t at = row * D;
    V xr[NC], yr[NC], gr[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t e = at + cl.col[c];
      xr[c] = V{};
      yr[c] = xr[c];
      gr[c] = xr[c];
      if (live && cl.some[c]) {
        xr[c] = load_vec<W, T, ONCE>(x + e, cl.width);
        if (y) yr[c] = load_vec<W, T, ONCE>(y + e, cl.width);
        if (a.gate_kind == EMB_GATE_ROWS) gr[c] = load_vec<W, T, ONCE>(gate + e, cl.width);
      }
    }
    float inv_y = 1.f;
    if (y && a.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) s[0] += squares<W>(wide<T>(yr[c]), cl.twice[c]);
      row_sums<TPR, 1>(s, lds, turn);
      turn ^= 1;
      inv_y = rsqrtf(s[0] * inv_d + a.eps);
    } else if (TPR > 64) {
      __syncthreads();  // r may be x's buffer: what two waves have is read by both before it is written
    }
    F rr[NC];
    float s[1] = {0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      rr[c] = a.alpha * wide<T>(xr[c]);
      if (y) {
        F v = wide<T>(yr[c]) * inv_y * wg[c];
        if (a.gate_kind == EMB_GATE_ROWS) v *= wide<T>(gr[c]);
        rr[c] += v;
      }
      s[0] += squares<W>(rr[c], cl.twice[c]);
    }
    if (r && live) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (cl.some[c]) store_vec<W, T, ONCE>(r + at + cl.col[c], rr[c], cl.width);
    }
    if (h) {
      row_sums<TPR, 1>(s, lds, turn);
      turn ^= 1;
      const float inv_r = rsqrtf(s[0] * inv_d + a.eps);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (live && cl.some[c]) store_vec<W, T, ONCE>(h + at + cl.col[c], rr[c] * inv_r * wp[c], cl.width);
    }
  }
}

// Rows go round the blocks; a thread keeps the column sums of its columns over the rows it sees in
// registers, the block's rows then meet in LDS, and the blocks in norm_join.  20011 x 2048 in bf16: 88 us,
// 5.6 TB/s; 5003 x 333 in fp32: 14.7 us.
template <typename T, int TPR, int NC, bool ONCE>
__global__ void __launch_bounds__(kThreads) norm_bwd(NormArgs a) {
  constexpr int kRows = kThreads / TPR, W = kVec<T>;
  typedef Vec<T, W> V;
  typedef Vec<float, W> F;
  constexpr int kSums = 6;
  __shared__ float lds[2][kThreads / 64][kSums];
  __shared__ __attribute__((aligned(16))) float cols[kRows > 1 ? kRows : 1][kRows > 1 ? TPR * W : 4];
  const int lane = threadIdx.x % TPR;
  const int D = a.dim;
  const T* r = static_cast<const T*>(a.r_in);
  const T* y = static_cast<const T*>(a.y);
  const T* gate = static_cast<const T*>(a.gate);
  const T* dr = static_cast<const T*>(a.dr);
  const T* dh = static_cast<const T*>(a.dh);
  T* dx = static_cast<T*>(a.dx);
  T* dy = static_cast<T*>(a.dy);
  T* dgate = a.gate_kind == EMB_GATE_ROWS ? static_cast<T*>(a.dgate) : nullptr;
  const float inv_d = 1.f / (float)D;
  const bool pre = a.w_pre != nullptr;

  const Columns<W, TPR, NC> cl(D, lane);
  F wg[NC], wp[NC], c_post[NC], c_pre[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    wg[c] = F(1.f);
    wp[c] = wg[c];
    c_post[c] = F{};
    c_pre[c] = F{};
    if (cl.some[c]) {
      if (a.w_post) wg[c] = load_vec<W>(a.w_post + cl.col[c], cl.width);
      if (a.gate_kind == EMB_GATE_VECTOR) wg[c] *= wide<T>(load_vec<W>(gate + cl.col[c], cl.width));
      if (pre) wp[c] = load_vec<W>(a.w_pre + cl.col[c], cl.width);
    }
  }
  // A row's data as it is.  Rows of a wave or less are loaded while the row before is computed (5003 x 333
  // in fp32: 19.3 -> 16.8 us); rows of a whole block are better off with the registers (20011 x 2048 in
  // bf16: 93 us, 95 that way).
  constexpr bool kAhead = TPR <= 64;
  struct Row {
    V r, y, g, dr, dh;
  };
  auto load = [&](int64_t base, Row (&x)[NC]) {
    const int64_t row = base + threadIdx.x / TPR, at = row * D;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t e = at + cl.col[c];
      x[c] = Row{};
      if (row >= a.rows || !cl.some[c]) continue;
      if (pre) {
        x[c].r = load_vec<W, T, ONCE>(r + e, cl.width);
        x[c].dh = load_vec<W, T, ONCE>(dh + e, cl.width);
      }
      if (dr) x[c].dr = load_vec<W, T, ONCE>(dr + e, cl.width);
      if (y) x[c].y = load_vec<W, T, ONCE>(y + e, cl.width);
      if (a.gate_kind == EMB_GATE_ROWS) x[c].g = load_vec<W, T, ONCE>(gate + e, cl.width);
    }
  };
  int turn = 0;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  Row now[NC], next[NC];
  if (kAhead) load((int64_t)blockIdx.x * kRows, now);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride) {
    const int64_t row = base + threadIdx.x / TPR;
    const bool live = row < a.rows;
    const int64_t at = row * D;
    if (kAhead) load(base + stride, next);
    else load(base, now);
    // r^2, u r, y^2, a dr, a u, a r
    float s[kSums] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const F rv = wide<T>(now[c].r), u = wide<T>(now[c].dh) * wp[c], yv = wide<T>(now[c].y), dv = wide<T>(now[c].dr);
      F av = yv * wg[c];
      if (a.gate_kind == EMB_GATE_ROWS) av *= wide<T>(now[c].g);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i < W - 1 && i < cl.twice[c]) continue;
        s[0] += rv[i] * rv[i];
        s[1] += u[i] * rv[i];
        s[2] += yv[i] * yv[i];
        s[3] += av[i] * dv[i];
        s[4] += av[i] * u[i];
        s[5] += av[i] * rv[i];
      }
    }
    row_sums<TPR, kSums>(s, lds, turn);
    turn ^= 1;
    const float inv_r = pre ? rsqrtf(s[0] * inv_d + a.eps) : 0.f;
    // dR = dr + inv_r (u - back_r r) and dy = inv_y (z - back_y y): a cube of an inverse is zero for rows of
    // about 1e15, and infinite for rows of zeros with an eps below 1e-25
    const float back_r = s[1] * inv_r * inv_d * inv_r;
    float inv_y = 1.f, back_y = 0.f;
    if (a.w_post) {
      inv_y = rsqrtf(s[2] * inv_d + a.eps);
      back_y = (s[3] + inv_r * (s[4] - back_r * s[5])) * inv_y * inv_d * inv_y;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (!cl.some[c]) continue;
      const int64_t e = at + cl.col[c];
      const F rv = wide<T>(now[c].r), dhv = wide<T>(now[c].dh), yv = wide<T>(now[c].y);
      const F dR = wide<T>(now[c].dr) + inv_r * (dhv * wp[c] - back_r * rv);
      F z = dR * wg[c];
      F yn = yv * inv_y;
      if (a.gate_kind == EMB_GATE_ROWS) {
        if (dgate && live) {
          // wg is w_post alone here (or 1)
          store_vec<W, T, ONCE>(dgate + e, dR * yn * wg[c], cl.width);
        }
        const F g = wide<T>(now[c].g);
        z *= g;
        yn *= g;
      }
      c_post[c] += dR * yn;
      c_pre[c] += dhv * (rv * inv_r);
      if (live) {
        if (dx) store_vec<W, T, ONCE>(dx + e, a.alpha * dR, cl.width);
        if (dy) store_vec<W, T, ONCE>(dy + e, inv_y * (z - back_y * yv), cl.width);
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (kAhead) now[c] = next[c];
  }
  // the block's column sums, [2][D] of its own
  float* out = a.part + (size_t)blockIdx.x * 2 * D;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const F v = k ? c_pre[c] : c_post[c];
      if constexpr (kRows == 1) {
        if (cl.some[c]) store_vec<W>(out + (size_t)k * D + cl.col[c], v, cl.width);
      } else {
        __syncthreads();
        *reinterpret_cast<F*>(&cols[threadIdx.x / TPR][lane * W]) = v;
        __syncthreads();
        for (int x = threadIdx.x; x < TPR * W; x += kThreads) {
          float t = 0.f;
#pragma unroll
          for (int g = 0; g < kRows; ++g) t += cols[g][x];
          const int at = c * TPR * W + x / W * W, i = x % W;
          if (at < D && i < cl.width) out[(size_t)k * D + min(at, D - cl.width) + i] = t;
        }
      }
    }
  }
}

// Sums the blocks' column sums: 32 columns of one of the two a workgroup, 32 threads a column, in a
// fixed order.  768 blocks of 2048 columns: 4.7 us, of which a launch is most.
constexpr int kJoin = 1024;
template <typename T>
__global__ void __launch_bounds__(kJoin) norm_join(NormArgs a) {
  __shared__ float lds[32][33];
  const int x = threadIdx.x & 31, part = threadIdx.x >> 5, k = blockIdx.y;
  const int col = blockIdx.x * 32 + x;
  float t = 0.f;
  if (col < a.dim) {
#pragma unroll 8
    for (int b = part; b < a.blocks; b += 32) t += a.part[((size_t)b * 2 + k) * a.dim + col];
  }
  lds[part][x] = t;
  __syncthreads();
  if (part == 0 && col < a.dim) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += lds[i][x];
    if (k == 1) {
      if (a.dw_pre) a.dw_pre[col] = v;
    } else if (a.gate_kind == EMB_GATE_VECTOR) {
      // the sum is of dR * y * inv(y) alone: the gate and the weights are the same in every row
      if (a.dgate) static_cast<float*>(a.dgate)[col] = v * (a.w_post ? a.w_post[col] : 1.f);
      if (a.dw_post) a.dw_post[col] = v * (float)static_cast<const T*>(a.gate)[col];
    } else if (a.dw_post) {
      a.dw_post[col] = v;
    }
  }
}

// How many threads take a row of `dim` columns, and in how many vectors each.
struct RowShape {
  int threads, vectors;
};
RowShape row_shape(int32_t dim, int vec) {
  if (dim <= 8 * vec) return {8, 1};
  if (dim <= 16 * vec) return {16, 1};
  if (dim <= 32 * vec) return {32, 1};
  if (dim <= 64 * vec) return {64, 1};
  if (dim <= 64 * vec * 2) return {64, 2};
  if (dim <= 256 * vec) return {256, 1};
  if (dim <= 256 * vec * 2) return {256, 2};
  if (dim <= 256 * vec * 4) return {256, 4};
  return {256, 8};  // fp32 alone
}

template <typename T>
bool once(const NormArgs& a, int rows_of_data) {
  return a.rows * a.dim * (int64_t)sizeof(T) * rows_of_data > kOnceBytes;
}
// Blocks of the forward.  Loads of a block's turn wait for the stores of its turn before, so many blocks with
// few turns are better; but each loads the weights, which weighs more where a thread has more of a row.
// 24M elements in rows of 200 in fp32, 1024 / 2048 / 8192 / 16384 blocks: 70 / 79 / 71 / 66 us; 500 in fp16:
// 38 / 41 / 37 / 38; 8192 in fp16, 512 / 1024 / 2048 / 8192: 40 / 43 / 45 / 48.
template <typename T, int TPR, int NC>
void go_fwd(const NormArgs& a, hipStream_t st) {
  constexpr int kFloats = NC * kVec<T>;  // of a row, in a thread
  constexpr int64_t kMost = kFloats <= 4 ? 16384 : kFloats <= 8 ? 8192 : 512;
  const int64_t blocks = (a.rows + kThreads / TPR - 1) / (kThreads / TPR);
  const dim3 grid((unsigned)(blocks < kMost ? blocks : kMost)), block(kThreads);
  if (once<T>(a, 4)) hipLaunchKernelGGL((norm_fwd<T, TPR, NC, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((norm_fwd<T, TPR, NC, false>), grid, block, 0, st, a);
}
template <typename T, int TPR, int NC>
void go_bwd(const NormArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.blocks), block(kThreads);
  if (a.blocks && once<T>(a, 6)) hipLaunchKernelGGL((norm_bwd<T, TPR, NC, true>), grid, block, 0, st, a);
  else if (a.blocks) hipLaunchKernelGGL((norm_bwd<T, TPR, NC, false>), grid, block, 0, st, a);
  hipLaunchKernelGGL((norm_join<T>), dim3((unsigned)((a.dim + 31) / 32), 2), dim3(kJoin), 0, st, a);
}

template <typename T>
void pick(const NormArgs& a, bool bwd, hipStream_t st) {
#define GO(TPR, NC)                                                       \
  if (s.threads == TPR && s.vectors == NC)                                \
    return bwd ? go_bwd<T, TPR, NC>(a, st) : go_fwd<T, TPR, NC>(a, st)
  const RowShape s = row_shape(a.dim, kVec<T>);
  GO(8, 1);
  GO(16, 1);
  GO(32, 1);
  GO(64, 1);
  GO(64, 2);
  GO(256, 1);
  GO(256, 2);
  GO(256, 4);
  if constexpr (kVec<T> == 4) GO(256, 8);
#undef GO
}

void pick_type(const NormArgs& a, bool bwd, hipStream_t st) {
  if (a.dtype == EMB_F32) pick<float>(a, bwd, st);
  else if (a.dtype == EMB_F16) pick<_Float16>(a, bwd, st);
  else pick<__bf16>(a, bwd, st);
}

}  // namespace

// Blocks of the backward, at most what is resident at once, so that the last ones do not run alone; each
// writes and norm_join reads 8 dim bytes.  24M elements, 512 / 768 / 1024 blocks: rows of 300 in fp16 86 / 74 /
// 88 us, of 700 64 / 79 / 71, of 500 in fp32 108 / 121 / 115, of 16 in fp32, where a block's own sums
// are most of the end, 136 / 110 / 104; rows of 8192 in fp16, 256 / 512: 79 / 87.
int norm_bwd_blocks(int64_t rows, int32_t dim, int32_t dtype) {
  const int vec = dtype == EMB_F32 ? 4 : 8;
  const RowShape s = row_shape(dim, vec);
  const int floats = s.vectors * vec;
  const int64_t per = kThreads / s.threads;
  const int64_t most = s.threads == 8 || (vec == 8 && floats == 8) ? 768 : floats < 32 ? 512 : 256;
  const int64_t b = (rows + per - 1) / per;
  return (int)(b < most ? b : most);
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
  pick_type(a, false, st);
  return hipGetLastError();
}
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st) {
  pick_type(a, true, st);
  return hipGetLastError();
}

}  // namespace emb
