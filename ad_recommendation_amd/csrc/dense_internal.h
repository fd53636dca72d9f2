// Internal declarations shared by the dense side's host entry points (dense_host.cpp) and its gfx950
// kernels (dense_attn.hip, dense_shared.hip, dense_shared_bwd.hip, dense_cache.hip, dense_norm.hip,
// dense_adamw.hip).  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "emb_dense.h"

namespace emb {

// ---------------------------------------------------------------- attention
struct AttnArgs {
  EmbHeads q, k, v, out, dout, dq, dk, dv;
  const int32_t* off;  // training: offsets; decode: lengths
  float* lse;
  float* delta;        // backward: out . dout, [q_heads][n_tok]
  float* part;         // partial results of split work
  int64_t n_tok;       // decode: the cache's capacity
  int32_t n_seq;
  int32_t q_heads, kv_heads, dim, window, sinks, dtype;
  float scale;
};

struct AttnBwdPlan {
  size_t off_part, bytes;
};
AttnBwdPlan plan_attn_bwd(const EmbAttn& a, int64_t n_seq, int64_t n_tok);
struct AttnDecodePlan {
  int32_t waves;   // of a workgroup
  int32_t splits;  // of a sequence's visible keys
  size_t bytes;
};
AttnDecodePlan plan_attn_decode(const EmbAttn& a, int64_t n_seq, int64_t capacity);

// Threads of a call's largest launch, of which there have to be fewer than 2^32.
int64_t attn_fwd_threads(const AttnArgs& a);
int64_t attn_bwd_threads(const AttnArgs& a);
int64_t attn_decode_threads(const AttnArgs& a, const AttnDecodePlan& p);

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t st);
hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t st);
hipError_t launch_attn_decode(const AttnArgs& a, const AttnDecodePlan& p, hipStream_t st);

// ---------------------------------------------------------------- attention of candidates
// What a query row sees of its request's own tokens: nothing (a newest event, which is cached), its token
// alone, or its candidate's tokens up to its own.
enum { kOwnNone, kOwnSelf, kOwnTiles };
struct SharedArgs : AttnArgs {  // off: tokens of requests, null for one token each
  EmbHeads hk, hv;              // history; in 8 bits its codes
  EmbHeads ke, ve;              // their exponents
  EmbHeads dhk, dhv;
  const int32_t* hist;          // packed: offsets of n_hist events; caches: lengths up to n_hist
  const int32_t* first;         // kOwnTiles
  float* self;                  // backward, kOwnSelf: p and ds of each row with itself, [2][q_heads][n_tok]
  int64_t n_hist;
  int32_t group;                // query heads of a key/value head
  int32_t back;                 // history events of the window
  int32_t packed, own;
};
struct SharedPlan {
  int32_t rows;    // of a tile: 32, whose keys the waves share out, or 128, 32 a wave
  int32_t waves;   // of 32 rows: of a workgroup
  int32_t splits;  // workgroups that may share a request's keys, so that each has `unit` tiles of them
  int32_t unit;
  size_t bytes;
};
// hist: events that a history has on average; most: that one may have.  one: one token a request, without offsets.
SharedPlan plan_shared(const EmbAttn& a, int64_t n_seq, int64_t n_tok, int64_t hist, int64_t most, bool one);
int64_t shared_threads(const SharedArgs& a, const SharedPlan& p);
hipError_t launch_shared(const SharedArgs& a, const SharedPlan& p, bool q8, hipStream_t st);

struct SharedBwdPlan {
  int32_t rows, splits, unit;  // of dq, as the forward's
  size_t off_self, off_part, bytes;
};
SharedBwdPlan plan_shared_bwd(const EmbAttn& a, int64_t n_seq, int64_t n_tok, int64_t n_hist);
int64_t shared_bwd_threads(const SharedArgs& a, const SharedBwdPlan& p);
hipError_t launch_shared_bwd(const SharedArgs& a, const SharedBwdPlan& p, hipStream_t st);

// ---------------------------------------------------------------- caches in 8 bits
struct CacheArgs {
  EmbHeads x[2];       // keys and values of packed tokens
  EmbHeads code[2], exp[2];
  const int32_t* off;  // null: one token a sequence
  const int32_t* start;  // null: 0
  int64_t n_tok, capacity;
  int32_t n_seq, heads, dim, dtype;
};
int64_t cache_threads(const CacheArgs& a);
hipError_t launch_cache(const CacheArgs& a, bool write, hipStream_t st);

// ---------------------------------------------------------------- norms
struct NormArgs {
  const void *x, *y, *gate;
  const float *w_post, *w_pre;
  const void *r_in, *dr, *dh;
  void *r, *h, *dx, *dy, *dgate;
  float *dw_post, *dw_pre;
  float* part;  // [blocks][2][dim]
  int64_t rows;
  int32_t dim, gate_kind, dtype, blocks;
  float alpha, eps;
};
int norm_bwd_blocks(int64_t rows, int32_t dim, int32_t dtype);
hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st);

// ---------------------------------------------------------------- AdamW
// One launch's tensors travel in the kernel's argument block (4 KiB at most), so a step needs no
// table in device memory and no copy, and is captured into a graph as it is.
struct AdamTensor {
  float* w;
  const void* g;
  void* copy;
  uint32_t n;
  uint32_t block0;  // first block of EMB_ADAMW_BLOCK elements in the state arrays
  uint32_t chunk0;  // first work chunk
  float wd;
};
constexpr int kAdamMax = 96;
// Elements of a workgroup: what its threads hold at once.  With more, taken in turn, the loads of a turn
// wait for the stores of the one before: 20.8M elements in fp32 97 us, 8192 a workgroup 115; 335.6M with
// 8-bit states 994, 8192 a workgroup 1.5 % more.
constexpr int kAdamChunk = 2048;
constexpr uint32_t kAdamChunks = 1 << 23;  // of a launch, which has fewer than 2^32 threads
struct AdamArgs {
  AdamTensor t[kAdamMax];
  float *m, *v;
  uint8_t *m8, *m_exp, *v8, *v_exp;
  const float* grad_scale;
  float lr, b1, b2, omb1, omb2, inv_c1, inv_c2, eps;
  uint32_t seed_lo, seed_hi, n_tensors;
  uint32_t once;  // more data than the caches hold
};
static_assert(sizeof(AdamArgs) <= 4096, "the argument block of a launch");
// elems: of the whole call, which may be several launches.
hipError_t launch_adamw(AdamArgs& a, int64_t elems, uint32_t n_chunks, bool q8, int grad_dtype,
                        int copy_dtype, hipStream_t st);
hipError_t launch_adamw_values(const uint8_t* codes, const uint8_t* exp, int64_t elems, void* out,
                               int out_dtype, hipStream_t st);

}  // namespace emb
