// C entry points of the dense side: argument checks, workspace sizes, launches.
#include "emb_dense.h"

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <string>
#include <utility>
#include <vector>

#include "dense_internal.h"
#include "emb_internal.h"

using namespace emb;

namespace {

#define DENSE_CHECK(cond, code, msg)                  \
  do {                                                \
    if (!(cond)) return set_error(code, msg);         \
  } while (0)

#define DENSE_TRY(expr)              \
  do {                               \
    const int rc_ = (expr);          \
    if (rc_ != EMB_OK) return rc_;   \
  } while (0)

// The failed call's code must not stay behind as the thread's last error (see emb_host.cpp).
int done(hipError_t e, const char* what) {
  if (e == hipSuccess) return EMB_OK;
  (void)hipGetLastError();
  return set_error(EMB_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int32_t t) { return t == EMB_F32 || t == EMB_F16 || t == EMB_BF16; }
size_t elem_bytes(int32_t t) { return t == EMB_F32 ? 4 : 2; }

bool validate_on() {
  const char* e = std::getenv("EMB_VALIDATE");
  return e && *e && std::strcmp(e, "0") != 0;
}

// ---------------------------------------------------------------- attention
int check_attn(const EmbAttn* a) {
  DENSE_CHECK(a, EMB_EINVAL, "attention: null descriptor");
  DENSE_CHECK(a->dtype == EMB_F16 || a->dtype == EMB_BF16, EMB_EINVAL,
              "attention: dtype must be EMB_F16 or EMB_BF16");
  DENSE_CHECK(a->kv_heads >= 1 && a->q_heads >= 1 && a->q_heads % a->kv_heads == 0, EMB_EINVAL,
              "attention: q_heads must be a positive multiple of kv_heads");
  DENSE_CHECK(a->q_heads <= 4096, EMB_ERANGE, "attention: more than 4096 query heads");
  DENSE_CHECK(a->dim >= 8 && a->dim <= 128 && a->dim % 8 == 0, EMB_EINVAL,
              "attention: dim must be a multiple of 8 from 8 to 128");
  DENSE_CHECK(a->window >= 1, EMB_EINVAL, "attention: window must be at least 1");
  DENSE_CHECK(a->sinks >= 0 && a->sinks <= EMB_ATTN_MAX_SINKS, EMB_EINVAL,
              "attention: sinks must lie in [0, EMB_ATTN_MAX_SINKS]");
  DENSE_CHECK(std::isfinite(a->scale), EMB_EINVAL, "attention: scale is not finite");
  return EMB_OK;
}

int check_heads(const EmbHeads* t, const char* name) {
  DENSE_CHECK(t && t->p, EMB_EINVAL, std::string("attention: null pointer: ") + name);
  DENSE_CHECK(aligned(t->p, 16), EMB_EINVAL,
              std::string("attention: not 16-byte aligned: ") + name);
  DENSE_CHECK(t->seq % 8 == 0 && t->tok % 8 == 0 && t->head % 8 == 0, EMB_EINVAL,
              std::string("attention: a stride is not a multiple of 8: ") + name);
  return EMB_OK;
}

// Of an output: no element may have two places in the tensor, of which the last written would win.
int check_written(const EmbHeads* t, int64_t tokens, int32_t heads, int32_t dim, const char* name) {
  DENSE_TRY(check_heads(t, name));
  const auto apart = [&](int64_t stride, int64_t n) { return n <= 1 || stride >= dim || stride <= -dim; };
  DENSE_CHECK(apart(t->tok, tokens) && apart(t->head, heads), EMB_EINVAL,
              std::string("attention: tokens or heads of an output overlap: ") + name);
  return EMB_OK;
}

// Of an output with three strides: that no two of its places are one. Every stride has to pass what the smaller
// ones span.
int check_apart(const EmbHeads* t, int64_t n_seq, int64_t tokens, int64_t heads, int64_t dim, const std::string& name) {
  const auto size = [](int64_t x) { return x >= 0 ? x : x > -INT64_MAX ? -x : INT64_MAX; };
  std::pair<int64_t, int64_t> by[3] = {{size(t->seq), n_seq}, {size(t->tok), tokens}, {size(t->head), heads}};
  std::sort(by, by + 3);
  int64_t span = dim;
  for (const auto& x : by) {
    if (x.second <= 1) continue;
    DENSE_CHECK(x.first >= span, EMB_EINVAL, "attention: places of an output overlap: " + name);
    // past 2^62 nothing else fits between
    span = x.first > ((int64_t)1 << 62) / x.second ? INT64_MAX : span + (x.second - 1) * x.first;
  }
  return EMB_OK;
}

int check_counts(int64_t n_seq, int64_t n_tok) {
  DENSE_CHECK(n_seq >= 0 && n_tok >= 0, EMB_EINVAL, "attention: negative size");
  // the kernels count tokens in 32 bits, with tiles past the last one
  DENSE_CHECK(n_seq <= (1 << 30) && n_tok <= (1 << 30), EMB_ERANGE,
              "attention: more than 2^30 sequences or tokens");
  return EMB_OK;
}

int check_launch(int64_t threads) {
  DENSE_CHECK(threads <= (int64_t)UINT32_MAX, EMB_ERANGE, "attention: more tiles than one launch holds");
  return EMB_OK;
}

// EMB_VALIDATE=1: the offsets (or lengths) as the device holds them.
// whole: the last one has to be n_tok, and not less.
int validate_offsets(const int32_t* d, int64_t n_seq, int64_t n_tok, bool lens, hipStream_t st, bool whole = true) {
  if (!validate_on()) return EMB_OK;
  try {
    std::vector<int32_t> h((size_t)n_seq + (lens ? 0 : 1));
    hipError_t e = hipMemcpyAsync(h.data(), d, h.size() * 4, hipMemcpyDeviceToHost, st);
    if (e == hipSuccess) e = hipStreamSynchronize(st);
    if (e != hipSuccess) return done(e, "attention: reading the offsets");
    if (lens) {
      for (int32_t x : h)
        DENSE_CHECK(x >= 0 && x <= n_tok, EMB_EINVAL, "attention: a length outside the cache");
      return EMB_OK;
    }
    DENSE_CHECK(h[0] == 0, EMB_EINVAL, "attention: offsets[0] != 0");
    for (size_t i = 1; i < h.size(); ++i)
      DENSE_CHECK(h[i] >= h[i - 1], EMB_EINVAL, "attention: offsets decrease");
    DENSE_CHECK(whole ? h.back() == n_tok : h.back() <= n_tok, EMB_EINVAL,
                whole ? "attention: offsets[n_seq] != n_tok" : "attention: offsets[n_seq] > n_tok");
  } catch (const std::bad_alloc&) {
    return set_error(EMB_ENOMEM, "attention: host memory");
  }
  return EMB_OK;
}

AttnArgs attn_args(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                   const int32_t* off, int64_t n_seq, int64_t n_tok) {
  AttnArgs x{};
  x.q = *q;
  x.k = *k;
  x.v = *v;
  x.off = off;
  x.n_seq = (int32_t)n_seq;
  x.n_tok = n_tok;
  x.q_heads = a->q_heads;
  x.kv_heads = a->kv_heads;
  x.dim = a->dim;
  x.window = a->window;
  x.sinks = a->sinks;
  x.dtype = a->dtype;
  x.scale = a->scale;
  return x;
}

// ---------------------------------------------------------------- caches in 8 bits
int check_codes(const EmbHeads* t, const EmbHeads* e, const char* name) {
  DENSE_CHECK(t && t->p && e && e->p, EMB_EINVAL, std::string("cache: null pointer: ") + name);
  DENSE_CHECK(aligned(t->p, 8) && t->seq % 8 == 0 && t->tok % 8 == 0 && t->head % 8 == 0, EMB_EINVAL,
              std::string("cache: codes not 8-byte aligned, or a stride no multiple of 8: ") + name);
  return EMB_OK;
}

// ---------------------------------------------------------------- attention of candidates
// The tokens of requests and what they see of their own.
struct SharedCall {
  const EmbAttn* a;
  const EmbHeads *q, *k, *v;
  const int32_t *off, *first;
  int64_t n_seq, n_tok;
};
// The checks that every form has in common.
int check_shared(const SharedCall& c) {
  DENSE_TRY(check_heads(c.q, "q"));
  DENSE_TRY(check_heads(c.k, "k"));
  DENSE_TRY(check_heads(c.v, "v"));
  DENSE_CHECK(c.off, EMB_EINVAL, "attention: null pointer: offsets");
  DENSE_CHECK(aligned(c.off, 4) && aligned(c.first, 4), EMB_EINVAL, "attention: offsets or first not 4-byte aligned");
  return EMB_OK;
}
SharedArgs shared_args(const SharedCall& c) {
  SharedArgs x{};
  static_cast<AttnArgs&>(x) = attn_args(c.a, c.q, c.k ? c.k : c.q, c.v ? c.v : c.q, c.off, c.n_seq, c.n_tok);
  x.group = c.a->q_heads / c.a->kv_heads;
  x.first = c.first;
  x.own = c.first ? kOwnTiles : kOwnSelf;
  x.back = c.a->window - 1;  // a candidate's place is the one after the last event
  return x;
}
// EMB_VALIDATE=1: that `first` names a candidate's first token for each token.
int validate_first(const SharedCall& c, hipStream_t st) {
  if (!validate_on() || !c.first) return EMB_OK;
  try {
    std::vector<int32_t> f((size_t)c.n_tok), off((size_t)c.n_seq + 1);
    hipError_t e = hipMemcpyAsync(f.data(), c.first, f.size() * 4, hipMemcpyDeviceToHost, st);
    if (e == hipSuccess) e = hipMemcpyAsync(off.data(), c.off, off.size() * 4, hipMemcpyDeviceToHost, st);
    if (e == hipSuccess) e = hipStreamSynchronize(st);
    if (e != hipSuccess) return done(e, "attention: reading first");
    for (int64_t s = 0; s < c.n_seq; ++s) {
      for (int64_t i = off[s]; i < off[s + 1]; ++i) {
        DENSE_CHECK(f[i] >= off[s] && f[i] <= i && f[f[i]] == f[i] && (i == off[s] || f[i] == i || f[i] == f[i - 1]),
                    EMB_EINVAL, "attention: first does not name the first token of a candidate");
      }
    }
  } catch (const std::bad_alloc&) {
    return set_error(EMB_ENOMEM, "attention: host memory");
  }
  return EMB_OK;
}

// What is known of histories: their mean, and of caches how long they may be.  A packed one over four times the
// mean is shared out as one of four times is.
SharedPlan packed_plan(const EmbAttn& a, int64_t n_seq, int64_t n_tok, int64_t n_hist) {
  const int64_t mean = (n_hist + std::max<int64_t>(n_seq, 1) - 1) / std::max<int64_t>(n_seq, 1);
  return plan_shared(a, n_seq, n_tok, mean, std::min(4 * mean, n_hist), false);
}
SharedPlan cache_plan(const EmbAttn& a, int64_t n_seq, int64_t n_tok, int64_t capacity) {
  return plan_shared(a, n_seq, n_tok, capacity / 2, capacity, false);
}

// The serving forms: histories are caches, in 16 bits or (k_exp) in 8.
int shared_cache(const SharedCall& c, const EmbHeads* hk, const EmbHeads* ke, const EmbHeads* hv, const EmbHeads* ve,
                 const int32_t* d_lens, int64_t capacity, bool q8, const EmbHeads* out, void* d_ws, size_t ws_bytes,
                 emb_stream_t stream, const char* what) {
  DENSE_TRY(check_attn(c.a));
  DENSE_TRY(check_counts(c.n_seq, c.n_tok));
  DENSE_TRY(check_counts(c.n_seq, capacity));
  if (c.n_seq == 0 || c.n_tok == 0) return EMB_OK;
  DENSE_TRY(check_shared(c));
  DENSE_TRY(check_written(out, c.n_tok, c.a->q_heads, c.a->dim, "out"));
  EmbHeads one = *out;
  one.seq = 0;
  DENSE_TRY(check_apart(&one, 1, c.n_tok, c.a->q_heads, c.a->dim, "out"));
  DENSE_CHECK(hk && hv && (!q8 || (ke && ve)), EMB_EINVAL, "attention: null pointer: cache");
  if (capacity > 0) {  // an empty cache has nothing to point at
    if (q8) {
      DENSE_TRY(check_codes(hk, ke, "k_cache"));
      DENSE_TRY(check_codes(hv, ve, "v_cache"));
    } else {
      DENSE_TRY(check_heads(hk, "k_cache"));
      DENSE_TRY(check_heads(hv, "v_cache"));
    }
  }
  DENSE_CHECK(d_lens, EMB_EINVAL, "attention: null pointer: lens");
  DENSE_CHECK(aligned(d_lens, 4), EMB_EINVAL, "attention: lens not 4-byte aligned");
  SharedArgs x = shared_args(c);
  x.hk = *hk;
  x.hv = *hv;
  if (q8) {
    x.ke = *ke;
    x.ve = *ve;
  }
  x.hist = d_lens;
  x.n_hist = capacity;
  const SharedPlan p = cache_plan(*c.a, c.n_seq, c.n_tok, capacity);
  DENSE_TRY(check_launch(shared_threads(x, p)));
  DENSE_CHECK(ws_bytes >= p.bytes, EMB_ENOSPACE, "attention: workspace too small");
  DENSE_CHECK(p.bytes == 0 || (d_ws && aligned(d_ws, 16)), EMB_EINVAL, "attention: null or misaligned workspace");
  hipStream_t st = static_cast<hipStream_t>(stream);
  DENSE_TRY(validate_offsets(c.off, c.n_seq, c.n_tok, false, st, false));
  DENSE_TRY(validate_offsets(d_lens, c.n_seq, capacity, true, st));
  DENSE_TRY(validate_first(c, st));
  x.out = *out;
  x.part = static_cast<float*>(d_ws);
  return done(launch_shared(x, p, q8, st), what);
}

// The training forms' checks of packed histories.
int check_packed(const SharedCall& c, const EmbHeads* hk, const EmbHeads* hv, const int32_t* hist_off, int64_t n_hist) {
  DENSE_TRY(check_shared(c));
  if (n_hist > 0) {
    DENSE_TRY(check_heads(hk, "hist_k"));
    DENSE_TRY(check_heads(hv, "hist_v"));
  } else {
    DENSE_CHECK(hk && hv, EMB_EINVAL, "attention: null pointer: history");
  }
  DENSE_CHECK(hist_off, EMB_EINVAL, "attention: null pointer: hist_offsets");
  DENSE_CHECK(aligned(hist_off, 4), EMB_EINVAL, "attention: hist_offsets not 4-byte aligned");
  return EMB_OK;
}
SharedArgs packed_args(const SharedCall& c, const EmbHeads* hk, const EmbHeads* hv, const int32_t* hist_off,
                       int64_t n_hist) {
  SharedArgs x = shared_args(c);
  x.hk = *hk;
  x.hv = *hv;
  x.hist = hist_off;
  x.n_hist = n_hist;
  x.packed = 1;
  return x;
}
int cache_call(int32_t kv_heads, int32_t dim, int32_t dtype, const EmbHeads* k, const EmbHeads* v,
               const int32_t* d_offsets, const int32_t* d_start, int64_t n_seq, int64_t n_tok, const EmbHeads* kc,
               const EmbHeads* ke, const EmbHeads* vc, const EmbHeads* ve, int64_t capacity, bool write,
               hipStream_t st, const char* what) {
  DENSE_CHECK(dtype_ok(dtype), EMB_EINVAL, "cache: bad dtype");
  DENSE_CHECK(kv_heads >= 1 && kv_heads <= 4096, EMB_EINVAL, "cache: kv_heads must lie in [1, 4096]");
  DENSE_CHECK(dim >= 8 && dim <= 128 && dim % 8 == 0, EMB_EINVAL, "cache: dim must be a multiple of 8 from 8 to 128");
  DENSE_TRY(check_counts(n_seq, n_tok));
  DENSE_TRY(check_counts(n_seq, capacity));
  if (n_seq == 0 || n_tok == 0 || (write && capacity == 0)) return EMB_OK;
  DENSE_TRY(check_heads(k, "k"));
  DENSE_TRY(check_heads(v, "v"));
  if (capacity > 0) {
    DENSE_TRY(check_codes(kc, ke, "k_cache"));
    DENSE_TRY(check_codes(vc, ve, "v_cache"));
  } else {
    DENSE_CHECK(kc && ke && vc && ve, EMB_EINVAL, "cache: null pointer: cache");
  }
  if (write) {
    DENSE_TRY(check_apart(kc, n_seq, capacity, kv_heads, dim, "k_cache"));
    DENSE_TRY(check_apart(vc, n_seq, capacity, kv_heads, dim, "v_cache"));
    DENSE_TRY(check_apart(ke, n_seq, capacity, kv_heads, 1, "k_exp"));
    DENSE_TRY(check_apart(ve, n_seq, capacity, kv_heads, 1, "v_exp"));
  } else {
    for (const EmbHeads* t : {k, v}) {
      EmbHeads one = *t;
      one.seq = 0;
      DENSE_TRY(check_apart(&one, 1, n_tok, kv_heads, dim, t == k ? "k" : "v"));
    }
  }
  DENSE_CHECK(d_offsets || n_tok == n_seq, EMB_EINVAL, "cache: without offsets every sequence has one token");
  DENSE_CHECK(aligned(d_offsets, 4) && aligned(d_start, 4), EMB_EINVAL, "cache: offsets or start not 4-byte aligned");
  CacheArgs x{};
  x.x[0] = *k;
  x.x[1] = *v;
  x.code[0] = *kc;
  x.code[1] = *vc;
  x.exp[0] = *ke;
  x.exp[1] = *ve;
  x.off = d_offsets;
  x.start = d_start;
  x.n_tok = n_tok;
  x.capacity = capacity;
  x.n_seq = (int32_t)n_seq;
  x.heads = kv_heads;
  x.dim = dim;
  x.dtype = dtype;
  DENSE_TRY(check_launch(cache_threads(x)));
  if (d_offsets) DENSE_TRY(validate_offsets(d_offsets, n_seq, n_tok, false, st, false));
  return done(launch_cache(x, write, st), what);
}

// ---------------------------------------------------------------- AdamW
struct AdamCall {
  int32_t n_tensors;
  const int64_t* n;
  void* const* w;
  const void* const* grads;
  int32_t grad_dtype;
  void* const* copies;
  int32_t copy_dtype;
  int64_t state_elems, step;
  double lr, b1, b2, eps;
  const float* wd;
  const float* scale;
};

int64_t padded(int64_t n) { return (n + EMB_ADAMW_BLOCK - 1) / EMB_ADAMW_BLOCK * EMB_ADAMW_BLOCK; }

int run_adamw(const AdamCall& c, AdamArgs& a, bool q8, hipStream_t st) {
  DENSE_CHECK(c.n_tensors >= 0, EMB_EINVAL, "adamw: negative count");
  DENSE_CHECK(c.n_tensors == 0 || (c.n && c.w && c.grads && c.wd), EMB_EINVAL,
              "adamw: null pointer");
  DENSE_CHECK(dtype_ok(c.grad_dtype), EMB_EINVAL, "adamw: bad gradient dtype");
  DENSE_CHECK(!c.copies || c.copy_dtype == EMB_F16 || c.copy_dtype == EMB_BF16, EMB_EINVAL,
              "adamw: copies must be EMB_F16 or EMB_BF16");
  DENSE_CHECK(c.step >= 1, EMB_EINVAL, "adamw: step must be at least 1");
  DENSE_CHECK(c.b1 >= 0. && c.b1 < 1. && c.b2 >= 0. && c.b2 < 1., EMB_EINVAL,
              "adamw: a beta lies outside [0, 1)");
  DENSE_CHECK((float)c.eps > 0.f && std::isfinite((float)c.eps) && std::isfinite((float)c.lr), EMB_EINVAL,
              "adamw: eps must be positive and lr finite");
  DENSE_CHECK(aligned(c.scale, 4), EMB_EINVAL, "adamw: misaligned gradient scale");
  int64_t total = 0;
  for (int32_t i = 0; i < c.n_tensors; ++i) {
    DENSE_CHECK(c.n[i] >= 0, EMB_EINVAL, "adamw: negative tensor size");
    DENSE_CHECK(c.n[i] <= (int64_t)UINT32_MAX, EMB_ERANGE, "adamw: a tensor of 2^32 elements or more");
    DENSE_CHECK(std::isfinite(c.wd[i]), EMB_EINVAL, "adamw: weight decay is not finite");
    total += padded(c.n[i]);
    DENSE_CHECK(total / EMB_ADAMW_BLOCK <= (int64_t)UINT32_MAX, EMB_ERANGE,
                "adamw: more than 2^39 state elements");
    if (c.n[i] == 0) continue;
    DENSE_CHECK(c.w[i] && c.grads[i] && (!c.copies || c.copies[i]), EMB_EINVAL,
                "adamw: null tensor");
    DENSE_CHECK(aligned(c.w[i], 4) && aligned(c.grads[i], elem_bytes(c.grad_dtype)) &&
                    (!c.copies || aligned(c.copies[i], 2)),
                EMB_EINVAL, "adamw: a tensor is not aligned to its elements");
  }
  DENSE_CHECK(total == c.state_elems, EMB_EINVAL,
              "adamw: the state arrays do not have adamw_state_elems elements");
  if (total == 0) return EMB_OK;

  a.lr = (float)c.lr;
  a.b1 = (float)c.b1;
  a.b2 = (float)c.b2;
  a.omb1 = (float)(1.0 - c.b1);
  a.omb2 = (float)(1.0 - c.b2);
  a.inv_c1 = (float)(1.0 / (1.0 - std::pow(c.b1, (double)c.step)));
  a.inv_c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(c.b2, (double)c.step)));
  a.eps = (float)c.eps;
  a.grad_scale = c.scale;
  uint32_t block0 = 0;
  int32_t i = 0;
  while (i < c.n_tensors) {
    uint32_t k = 0;
    uint64_t chunks = 0;
    for (; i < c.n_tensors && k < (uint32_t)kAdamMax && chunks < kAdamChunks; ++i) {
      if (c.n[i] == 0) continue;
      AdamTensor& t = a.t[k++];
      t.w = static_cast<float*>(c.w[i]);
      t.g = c.grads[i];
      t.copy = c.copies ? c.copies[i] : nullptr;
      t.n = (uint32_t)c.n[i];
      t.block0 = block0;
      t.chunk0 = (uint32_t)chunks;
      t.wd = c.wd[i];
      block0 += (uint32_t)(padded(c.n[i]) / EMB_ADAMW_BLOCK);
      chunks += ((uint64_t)c.n[i] + kAdamChunk - 1) / kAdamChunk;
    }
    if (k == 0) break;
    a.n_tensors = k;
    DENSE_TRY(done(launch_adamw(a, total, (uint32_t)chunks, q8, c.grad_dtype,
                                c.copies ? c.copy_dtype : -1, st),
                   "adamw"));
  }
  return EMB_OK;
}

}  // namespace

extern "C" {

int attn_window_fwd(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                    const int32_t* d_offsets, int64_t n_seq, int64_t n_tok, const EmbHeads* out,
                    float* d_lse, emb_stream_t stream) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, n_tok));
  if (n_seq == 0 || n_tok == 0) return EMB_OK;
  DENSE_TRY(check_heads(q, "q"));
  DENSE_TRY(check_heads(k, "k"));
  DENSE_TRY(check_heads(v, "v"));
  DENSE_TRY(check_written(out, n_tok, a->q_heads, a->dim, "out"));
  DENSE_CHECK(d_offsets, EMB_EINVAL, "attention: null pointer: offsets");
  DENSE_CHECK(aligned(d_offsets, 4) && aligned(d_lse, 4), EMB_EINVAL,
              "attention: offsets or lse not 4-byte aligned");
  AttnArgs x = attn_args(a, q, k, v, d_offsets, n_seq, n_tok);
  DENSE_TRY(check_launch(attn_fwd_threads(x)));
  hipStream_t st = static_cast<hipStream_t>(stream);
  DENSE_TRY(validate_offsets(d_offsets, n_seq, n_tok, false, st));
  x.out = *out;
  x.lse = d_lse;
  return done(launch_attn_fwd(x, st), "attn_window_fwd");
}

int attn_window_bwd_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t n_tok, size_t* bytes) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, n_tok));
  DENSE_CHECK(bytes, EMB_EINVAL, "attention: null pointer: bytes");
  *bytes = plan_attn_bwd(*a, n_seq, n_tok).bytes;
  return EMB_OK;
}

int attn_window_bwd(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                    const int32_t* d_offsets, int64_t n_seq, int64_t n_tok, const EmbHeads* out,
                    const float* d_lse, const EmbHeads* dout, const EmbHeads* dq,
                    const EmbHeads* dk, const EmbHeads* dv, void* d_ws, size_t ws_bytes,
                    emb_stream_t stream) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, n_tok));
  if (n_seq == 0 || n_tok == 0) return EMB_OK;
  DENSE_TRY(check_heads(q, "q"));
  DENSE_TRY(check_heads(k, "k"));
  DENSE_TRY(check_heads(v, "v"));
  DENSE_TRY(check_heads(out, "out"));
  DENSE_TRY(check_heads(dout, "dout"));
  DENSE_TRY(check_written(dq, n_tok, a->q_heads, a->dim, "dq"));
  DENSE_TRY(check_written(dk, n_tok, a->kv_heads, a->dim, "dk"));
  DENSE_TRY(check_written(dv, n_tok, a->kv_heads, a->dim, "dv"));
  DENSE_CHECK(d_offsets && d_lse && d_ws, EMB_EINVAL,
              "attention: null pointer: offsets, lse or workspace");
  DENSE_CHECK(aligned(d_offsets, 4) && aligned(d_lse, 4) && aligned(d_ws, 16), EMB_EINVAL,
              "attention: misaligned offsets, lse or workspace");
  AttnArgs x = attn_args(a, q, k, v, d_offsets, n_seq, n_tok);
  DENSE_TRY(check_launch(attn_bwd_threads(x)));
  const AttnBwdPlan p = plan_attn_bwd(*a, n_seq, n_tok);
  DENSE_CHECK(ws_bytes >= p.bytes, EMB_ENOSPACE, "attention: workspace too small");
  hipStream_t st = static_cast<hipStream_t>(stream);
  DENSE_TRY(validate_offsets(d_offsets, n_seq, n_tok, false, st));
  x.out = *out;
  x.lse = const_cast<float*>(d_lse);
  x.dout = *dout;
  x.dq = *dq;
  x.dk = *dk;
  x.dv = *dv;
  x.delta = static_cast<float*>(d_ws);
  x.part = reinterpret_cast<float*>(static_cast<char*>(d_ws) + p.off_part);
  return done(launch_attn_bwd(x, st), "attn_window_bwd");
}

int attn_window_decode_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t capacity,
                                       size_t* bytes) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, capacity));
  DENSE_CHECK(bytes, EMB_EINVAL, "attention: null pointer: bytes");
  *bytes = plan_attn_decode(*a, n_seq, capacity).bytes;
  return EMB_OK;
}

int attn_window_decode(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k_cache,
                       const EmbHeads* v_cache, const int32_t* d_lens, int64_t n_seq,
                       int64_t capacity, const EmbHeads* out, void* d_ws, size_t ws_bytes,
                       emb_stream_t stream) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, capacity));
  if (n_seq == 0) return EMB_OK;
  DENSE_TRY(check_heads(q, "q"));
  DENSE_TRY(check_written(out, n_seq, a->q_heads, a->dim, "out"));
  if (capacity > 0) {  // an empty cache has nothing to point at
    DENSE_TRY(check_heads(k_cache, "k_cache"));
    DENSE_TRY(check_heads(v_cache, "v_cache"));
  } else {
    DENSE_CHECK(k_cache && v_cache, EMB_EINVAL, "attention: null pointer: cache");
  }
  DENSE_CHECK(d_lens, EMB_EINVAL, "attention: null pointer: lens");
  DENSE_CHECK(aligned(d_lens, 4), EMB_EINVAL, "attention: lens not 4-byte aligned");
  const AttnDecodePlan p = plan_attn_decode(*a, n_seq, capacity);
  AttnArgs x = attn_args(a, q, k_cache, v_cache, d_lens, n_seq, capacity);
  DENSE_TRY(check_launch(attn_decode_threads(x, p)));
  DENSE_CHECK(ws_bytes >= p.bytes, EMB_ENOSPACE, "attention: workspace too small");
  DENSE_CHECK(p.bytes == 0 || (d_ws && aligned(d_ws, 16)), EMB_EINVAL,
              "attention: null or misaligned workspace");
  hipStream_t st = static_cast<hipStream_t>(stream);
  DENSE_TRY(validate_offsets(d_lens, n_seq, capacity, true, st));
  x.out = *out;
  x.part = static_cast<float*>(d_ws);
  return done(launch_attn_decode(x, p, st), "attn_window_decode");
}

int attn_window_decode_q8_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t capacity, size_t* bytes) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, capacity));
  DENSE_CHECK(bytes, EMB_EINVAL, "attention: null pointer: bytes");
  *bytes = plan_shared(*a, n_seq, n_seq, capacity, capacity, true).bytes;
  return EMB_OK;
}

int attn_window_decode_q8(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k_cache, const EmbHeads* k_exp,
                          const EmbHeads* v_cache, const EmbHeads* v_exp, const int32_t* d_lens, int64_t n_seq,
                          int64_t capacity, const EmbHeads* out, void* d_ws, size_t ws_bytes, emb_stream_t stream) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, capacity));
  if (n_seq == 0) return EMB_OK;
  DENSE_TRY(check_heads(q, "q"));
  DENSE_TRY(check_written(out, n_seq, a->q_heads, a->dim, "out"));
  EmbHeads one = *out;
  one.seq = 0;
  DENSE_TRY(check_apart(&one, 1, n_seq, a->q_heads, a->dim, "out"));
  DENSE_CHECK(k_cache && v_cache && k_exp && v_exp, EMB_EINVAL, "attention: null pointer: cache");
  if (capacity > 0) {  // an empty cache has nothing to point at
    DENSE_TRY(check_codes(k_cache, k_exp, "k_cache"));
    DENSE_TRY(check_codes(v_cache, v_exp, "v_cache"));
  }
  DENSE_CHECK(d_lens, EMB_EINVAL, "attention: null pointer: lens");
  DENSE_CHECK(aligned(d_lens, 4), EMB_EINVAL, "attention: lens not 4-byte aligned");
  SharedArgs x = shared_args({a, q, nullptr, nullptr, nullptr, nullptr, n_seq, n_seq});
  x.own = kOwnNone;
  x.back = a->window;  // the query is at the last cached event
  x.hk = *k_cache;
  x.hv = *v_cache;
  x.ke = *k_exp;
  x.ve = *v_exp;
  x.hist = d_lens;
  x.n_hist = capacity;
  const SharedPlan p = plan_shared(*a, n_seq, n_seq, capacity, capacity, true);
  DENSE_TRY(check_launch(shared_threads(x, p)));
  DENSE_CHECK(ws_bytes >= p.bytes, EMB_ENOSPACE, "attention: workspace too small");
  DENSE_CHECK(p.bytes == 0 || (d_ws && aligned(d_ws, 16)), EMB_EINVAL, "attention: null or misaligned workspace");
  hipStream_t st = static_cast<hipStream_t>(stream);
  DENSE_TRY(validate_offsets(d_lens, n_seq, capacity, true, st));
  x.out = *out;
  x.part = static_cast<float*>(d_ws);
  return done(launch_shared(x, p, true, st), "attn_window_decode_q8");
}

int attn_shared_fwd_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t n_tok, int64_t n_hist, size_t* bytes) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, n_tok));
  DENSE_TRY(check_counts(n_seq, n_hist));
  DENSE_CHECK(bytes, EMB_EINVAL, "attention: null pointer: bytes");
  *bytes = packed_plan(*a, n_seq, n_tok, n_hist).bytes;
  return EMB_OK;
}

int attn_shared_fwd(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v, const EmbHeads* hist_k,
                    const EmbHeads* hist_v, const int32_t* d_offsets, const int32_t* d_first,
                    const int32_t* d_hist_offsets, int64_t n_seq, int64_t n_tok, int64_t n_hist, const EmbHeads* out,
                    float* d_lse, void* d_ws, size_t ws_bytes, emb_stream_t stream) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, n_tok));
  DENSE_TRY(check_counts(n_seq, n_hist));
  if (n_seq == 0 || n_tok == 0) return EMB_OK;
  const SharedCall c{a, q, k, v, d_offsets, d_first, n_seq, n_tok};
  DENSE_TRY(check_packed(c, hist_k, hist_v, d_hist_offsets, n_hist));
  DENSE_TRY(check_written(out, n_tok, a->q_heads, a->dim, "out"));
  EmbHeads one = *out;
  one.seq = 0;
  DENSE_TRY(check_apart(&one, 1, n_tok, a->q_heads, a->dim, "out"));
  DENSE_CHECK(aligned(d_lse, 4), EMB_EINVAL, "attention: lse not 4-byte aligned");
  SharedArgs x = packed_args(c, hist_k, hist_v, d_hist_offsets, n_hist);
  const SharedPlan p = packed_plan(*a, n_seq, n_tok, n_hist);
  DENSE_TRY(check_launch(shared_threads(x, p)));
  DENSE_CHECK(ws_bytes >= p.bytes, EMB_ENOSPACE, "attention: workspace too small");
  DENSE_CHECK(p.bytes == 0 || (d_ws && aligned(d_ws, 16)), EMB_EINVAL, "attention: null or misaligned workspace");
  hipStream_t st = static_cast<hipStream_t>(stream);
  DENSE_TRY(validate_offsets(d_offsets, n_seq, n_tok, false, st, false));
  DENSE_TRY(validate_offsets(d_hist_offsets, n_seq, n_hist, false, st, false));
  DENSE_TRY(validate_first(c, st));
  x.out = *out;
  x.lse = d_lse;
  x.part = static_cast<float*>(d_ws);
  return done(launch_shared(x, p, false, st), "attn_shared_fwd");
}

int attn_shared_bwd_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t n_tok, int64_t n_hist, size_t* bytes) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, n_tok));
  DENSE_TRY(check_counts(n_seq, n_hist));
  DENSE_CHECK(bytes, EMB_EINVAL, "attention: null pointer: bytes");
  *bytes = plan_shared_bwd(*a, n_seq, n_tok, n_hist).bytes;
  return EMB_OK;
}

int attn_shared_bwd(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v, const EmbHeads* hist_k,
                    const EmbHeads* hist_v, const int32_t* d_offsets, const int32_t* d_first,
                    const int32_t* d_hist_offsets, int64_t n_seq, int64_t n_tok, int64_t n_hist, const EmbHeads* out,
                    const float* d_lse, const EmbHeads* dout, const EmbHeads* dq, const EmbHeads* dk,
                    const EmbHeads* dv, const EmbHeads* dhist_k, const EmbHeads* dhist_v, void* d_ws, size_t ws_bytes,
                    emb_stream_t stream) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, n_tok));
  DENSE_TRY(check_counts(n_seq, n_hist));
  if (n_seq == 0 || (n_tok == 0 && n_hist == 0)) return EMB_OK;
  const SharedCall c{a, q, k, v, d_offsets, d_first, n_seq, n_tok};
  // without tokens the history's gradients are zeros, and what the tokens' arrays point at is not read
  if (n_tok > 0) {
    DENSE_TRY(check_packed(c, hist_k, hist_v, d_hist_offsets, n_hist));
    DENSE_TRY(check_heads(out, "out"));
    DENSE_TRY(check_heads(dout, "dout"));
    DENSE_CHECK(d_lse && d_ws, EMB_EINVAL, "attention: null pointer: lse or workspace");
    DENSE_CHECK(aligned(d_lse, 4) && aligned(d_ws, 16), EMB_EINVAL, "attention: misaligned lse or workspace");
  } else {
    DENSE_CHECK(q && k && v && out && dout && dq && dk && dv && d_offsets && d_hist_offsets, EMB_EINVAL,
                "attention: null pointer");
    DENSE_TRY(check_heads(hist_k, "hist_k"));
    DENSE_TRY(check_heads(hist_v, "hist_v"));
    DENSE_CHECK(aligned(d_offsets, 4) && aligned(d_hist_offsets, 4), EMB_EINVAL, "attention: misaligned offsets");
  }
  const struct {
    const EmbHeads* t;
    int64_t n;
    int32_t heads;
    const char* name;
  } written[] = {{dq, n_tok, a->q_heads, "dq"},
                 {dk, n_tok, a->kv_heads, "dk"},
                 {dv, n_tok, a->kv_heads, "dv"},
                 {dhist_k, n_hist, a->kv_heads, "dhist_k"},
                 {dhist_v, n_hist, a->kv_heads, "dhist_v"}};
  for (const auto& w : written) {
    DENSE_CHECK(w.t, EMB_EINVAL, std::string("attention: null pointer: ") + w.name);
    if (w.n == 0) continue;
    DENSE_TRY(check_heads(w.t, w.name));
    EmbHeads one = *w.t;
    one.seq = 0;
    DENSE_TRY(check_apart(&one, 1, w.n, w.heads, a->dim, w.name));
  }
  SharedArgs x = packed_args(c, hist_k, hist_v, d_hist_offsets, n_hist);
  const SharedBwdPlan p = plan_shared_bwd(*a, n_seq, n_tok, n_hist);
  DENSE_TRY(check_launch(shared_bwd_threads(x, p)));
  DENSE_CHECK(ws_bytes >= p.bytes, EMB_ENOSPACE, "attention: workspace too small");
  hipStream_t st = static_cast<hipStream_t>(stream);
  DENSE_TRY(validate_offsets(d_offsets, n_seq, n_tok, false, st, false));
  DENSE_TRY(validate_offsets(d_hist_offsets, n_seq, n_hist, false, st, false));
  DENSE_TRY(validate_first(c, st));
  x.out = *out;
  x.lse = const_cast<float*>(d_lse);
  x.dout = *dout;
  x.dq = *dq;
  x.dk = *dk;
  x.dv = *dv;
  x.dhk = *dhist_k;
  x.dhv = *dhist_v;
  x.delta = static_cast<float*>(d_ws);
  x.self = reinterpret_cast<float*>(static_cast<char*>(d_ws) + p.off_self);
  x.part = reinterpret_cast<float*>(static_cast<char*>(d_ws) + p.off_part);
  return done(launch_shared_bwd(x, p, st), "attn_shared_bwd");
}

int attn_shared_cache_workspace_bytes(const EmbAttn* a, int64_t n_seq, int64_t n_tok, int64_t capacity, size_t* bytes) {
  DENSE_TRY(check_attn(a));
  DENSE_TRY(check_counts(n_seq, n_tok));
  DENSE_TRY(check_counts(n_seq, capacity));
  DENSE_CHECK(bytes, EMB_EINVAL, "attention: null pointer: bytes");
  *bytes = cache_plan(*a, n_seq, n_tok, capacity).bytes;
  return EMB_OK;
}

int attn_shared_cache(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                      const EmbHeads* k_cache, const EmbHeads* v_cache, const int32_t* d_offsets,
                      const int32_t* d_first, const int32_t* d_lens, int64_t n_seq, int64_t n_tok, int64_t capacity,
                      const EmbHeads* out, void* d_ws, size_t ws_bytes, emb_stream_t stream) {
  return shared_cache({a, q, k, v, d_offsets, d_first, n_seq, n_tok}, k_cache, nullptr, v_cache, nullptr, d_lens,
                      capacity, false, out, d_ws, ws_bytes, stream, "attn_shared_cache");
}

int attn_shared_cache_q8(const EmbAttn* a, const EmbHeads* q, const EmbHeads* k, const EmbHeads* v,
                         const EmbHeads* k_cache, const EmbHeads* k_exp, const EmbHeads* v_cache,
                         const EmbHeads* v_exp, const int32_t* d_offsets, const int32_t* d_first,
                         const int32_t* d_lens, int64_t n_seq, int64_t n_tok, int64_t capacity, const EmbHeads* out,
                         void* d_ws, size_t ws_bytes, emb_stream_t stream) {
  return shared_cache({a, q, k, v, d_offsets, d_first, n_seq, n_tok}, k_cache, k_exp, v_cache, v_exp, d_lens, capacity,
                      true, out, d_ws, ws_bytes, stream, "attn_shared_cache_q8");
}

int cache_q8_write(int32_t kv_heads, int32_t dim, int32_t dtype, const EmbHeads* k, const EmbHeads* v,
                   const int32_t* d_offsets, const int32_t* d_start, int64_t n_seq, int64_t n_tok,
                   const EmbHeads* k_cache, const EmbHeads* k_exp, const EmbHeads* v_cache, const EmbHeads* v_exp,
                   int64_t capacity, emb_stream_t stream) {
  return cache_call(kv_heads, dim, dtype, k, v, d_offsets, d_start, n_seq, n_tok, k_cache, k_exp, v_cache, v_exp,
                    capacity, true, static_cast<hipStream_t>(stream), "cache_q8_write");
}

int cache_q8_read(int32_t kv_heads, int32_t dim, int32_t dtype, const EmbHeads* k_cache, const EmbHeads* k_exp,
                  const EmbHeads* v_cache, const EmbHeads* v_exp, int64_t capacity, const int32_t* d_offsets,
                  const int32_t* d_start, int64_t n_seq, int64_t n_tok, const EmbHeads* k, const EmbHeads* v,
                  emb_stream_t stream) {
  return cache_call(kv_heads, dim, dtype, k, v, d_offsets, d_start, n_seq, n_tok, k_cache, k_exp, v_cache, v_exp,
                    capacity, false, static_cast<hipStream_t>(stream), "cache_q8_read");
}

static int check_norm(const void* y, const void* gate, int32_t gate_kind, const float* w_post,
                      const float* w_pre, int64_t rows, int32_t dim, int32_t dtype, float alpha,
                      float eps) {
  DENSE_CHECK(dtype_ok(dtype), EMB_EINVAL, "norm: bad dtype");
  DENSE_CHECK(dim >= 1 && dim <= 8192, EMB_EINVAL, "norm: dim must lie in [1, 8192]");
  DENSE_CHECK(rows >= 0, EMB_EINVAL, "norm: negative row count");
  DENSE_CHECK(rows <= ((int64_t)1 << 40), EMB_ERANGE, "norm: more than 2^40 rows");
  DENSE_CHECK(gate_kind >= EMB_GATE_NONE && gate_kind <= EMB_GATE_ROWS, EMB_EINVAL,
              "norm: bad gate kind");
  const bool gate_needed = gate_kind == EMB_GATE_VECTOR || (gate_kind == EMB_GATE_ROWS && rows > 0);
  DENSE_CHECK(gate_kind == EMB_GATE_NONE ? !gate : (gate || !gate_needed), EMB_EINVAL,
              "norm: gate and its kind disagree");
  DENSE_CHECK(y || rows == 0 || (gate_kind == EMB_GATE_NONE && !w_post), EMB_EINVAL,
              "norm: a gate or w_post without y");
  DENSE_CHECK(std::isfinite(alpha) && std::isfinite(eps) && eps > 0.f, EMB_EINVAL,
              "norm: alpha must be finite and eps positive");
  const size_t e = elem_bytes(dtype);
  DENSE_CHECK(aligned(y, e) && aligned(gate, e) && aligned(w_post, 4) && aligned(w_pre, 4),
              EMB_EINVAL, "norm: a tensor is not aligned to its elements");
  return EMB_OK;
}

int norm_gate_residual_fwd(const void* x, const void* y, const void* gate, int32_t gate_kind,
                           const float* w_post, const float* w_pre, int64_t rows, int32_t dim,
                           int32_t dtype, float alpha, float eps, void* r, void* h,
                           emb_stream_t stream) {
  DENSE_TRY(check_norm(y, gate, gate_kind, w_post, w_pre, rows, dim, dtype, alpha, eps));
  if (rows == 0) return EMB_OK;
  DENSE_CHECK(x, EMB_EINVAL, "norm: null pointer: x");
  DENSE_CHECK((w_pre != nullptr) == (h != nullptr), EMB_EINVAL, "norm: h goes with w_pre");
  DENSE_CHECK(r || h, EMB_EINVAL, "norm: neither r nor h");
  const size_t e = elem_bytes(dtype);
  DENSE_CHECK(aligned(x, e) && aligned(r, e) && aligned(h, e), EMB_EINVAL,
              "norm: a tensor is not aligned to its elements");
  NormArgs a{};
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.r = r;
  a.h = h;
  a.rows = rows;
  a.dim = dim;
  a.gate_kind = gate_kind;
  a.dtype = dtype;
  a.alpha = alpha;
  a.eps = eps;
  return done(launch_norm_fwd(a, static_cast<hipStream_t>(stream)), "norm_gate_residual_fwd");
}

int norm_gate_residual_bwd_workspace_bytes(int64_t rows, int32_t dim, size_t* bytes) {
  DENSE_CHECK(dim >= 1 && dim <= 8192, EMB_EINVAL, "norm: dim must lie in [1, 8192]");
  DENSE_CHECK(rows >= 0, EMB_EINVAL, "norm: negative row count");
  DENSE_CHECK(bytes, EMB_EINVAL, "norm: null pointer: bytes");
  const int blocks = std::max(norm_bwd_blocks(rows, dim, EMB_F32), norm_bwd_blocks(rows, dim, EMB_F16));
  *bytes = (size_t)blocks * 2 * (size_t)dim * sizeof(float);
  return EMB_OK;
}

int norm_gate_residual_bwd(const void* r, const void* y, const void* gate, int32_t gate_kind,
                           const float* w_post, const float* w_pre, int64_t rows, int32_t dim,
                           int32_t dtype, float alpha, float eps, const void* dr, const void* dh,
                           void* dx, void* dy, void* dgate, float* dw_post, float* dw_pre,
                           void* d_ws, size_t ws_bytes, emb_stream_t stream) {
  DENSE_TRY(check_norm(y, gate, gate_kind, w_post, w_pre, rows, dim, dtype, alpha, eps));
  DENSE_CHECK(rows == 0 || (dh != nullptr) == (w_pre != nullptr), EMB_EINVAL,
              "norm: dh goes with w_pre");
  DENSE_CHECK(rows == 0 || dr || dh, EMB_EINVAL, "norm: neither dr nor dh");
  DENSE_CHECK(rows == 0 || r || !w_pre, EMB_EINVAL, "norm: null pointer: r");
  DENSE_CHECK(!dy || y || rows == 0, EMB_EINVAL, "norm: dy without y");
  DENSE_CHECK(!dgate || gate_kind != EMB_GATE_NONE, EMB_EINVAL, "norm: dgate without a gate");
  DENSE_CHECK(!dw_post || w_post, EMB_EINVAL, "norm: dw_post without w_post");
  DENSE_CHECK(!dw_pre || w_pre, EMB_EINVAL, "norm: dw_pre without w_pre");
  const size_t e = elem_bytes(dtype);
  DENSE_CHECK(aligned(r, e) && aligned(dr, e) && aligned(dh, e) && aligned(dx, e) &&
                  aligned(dy, e) && aligned(dgate, gate_kind == EMB_GATE_VECTOR ? 4 : e) &&
                  aligned(dw_post, 4) && aligned(dw_pre, 4),
              EMB_EINVAL, "norm: a tensor is not aligned to its elements");
  NormArgs a{};
  a.blocks = norm_bwd_blocks(rows, dim, dtype);
  const size_t need = (size_t)a.blocks * 2 * (size_t)dim * sizeof(float);
  DENSE_CHECK(ws_bytes >= need, EMB_ENOSPACE, "norm: workspace too small");
  DENSE_CHECK(need == 0 || (d_ws && aligned(d_ws, 16)), EMB_EINVAL,
              "norm: null or misaligned workspace");
  a.y = y;
  a.gate = gate;
  a.w_post = w_post;
  a.w_pre = w_pre;
  a.r_in = r;
  a.dr = dr;
  a.dh = dh;
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.dw_post = dw_post;
  a.dw_pre = dw_pre;
  a.part = static_cast<float*>(d_ws);
  a.rows = rows;
  a.dim = dim;
  a.gate_kind = gate_kind;
  a.dtype = dtype;
  a.alpha = alpha;
  a.eps = eps;
  return done(launch_norm_bwd(a, static_cast<hipStream_t>(stream)), "norm_gate_residual_bwd");
}

int adamw_state_elems(const int64_t* n, int32_t n_tensors, int64_t* elems) {
  DENSE_CHECK(elems && n_tensors >= 0 && (n || n_tensors == 0), EMB_EINVAL, "adamw: null pointer");
  int64_t total = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    DENSE_CHECK(n[i] >= 0, EMB_EINVAL, "adamw: negative tensor size");
    DENSE_CHECK(n[i] <= (int64_t)UINT32_MAX, EMB_ERANGE, "adamw: a tensor of 2^32 elements or more");
    total += padded(n[i]);
  }
  *elems = total;
  return EMB_OK;
}

int adamw_step(int32_t n_tensors, const int64_t* n, void* const* w, const void* const* grads,
               int32_t grad_dtype, void* const* copies, int32_t copy_dtype, float* d_m, float* d_v,
               int64_t state_elems, int64_t step, double lr, double beta1, double beta2, double eps,
               const float* weight_decay, const float* d_grad_scale, emb_stream_t stream) {
  DENSE_CHECK(state_elems == 0 || (d_m && d_v), EMB_EINVAL, "adamw: null state");
  DENSE_CHECK(aligned(d_m, 16) && aligned(d_v, 16), EMB_EINVAL, "adamw: states not 16-byte aligned");
  AdamArgs a;
  std::memset(&a, 0, sizeof a);
  a.m = d_m;
  a.v = d_v;
  const AdamCall c{n_tensors, n, w, grads, grad_dtype, copies, copy_dtype, state_elems, step,
                   lr, beta1, beta2, eps, weight_decay, d_grad_scale};
  return run_adamw(c, a, false, static_cast<hipStream_t>(stream));
}

int adamw_step_q8(int32_t n_tensors, const int64_t* n, void* const* w, const void* const* grads,
                  int32_t grad_dtype, void* const* copies, int32_t copy_dtype, uint8_t* d_m,
                  uint8_t* d_m_exp, uint8_t* d_v, uint8_t* d_v_exp, int64_t state_elems,
                  int64_t step, double lr, double beta1, double beta2, double eps,
                  const float* weight_decay, const float* d_grad_scale, uint64_t seed,
                  emb_stream_t stream) {
  DENSE_CHECK(state_elems == 0 || (d_m && d_m_exp && d_v && d_v_exp), EMB_EINVAL,
              "adamw: null state");
  DENSE_CHECK(aligned(d_m, 16) && aligned(d_v, 16), EMB_EINVAL, "adamw: states not 16-byte aligned");
  AdamArgs a;
  std::memset(&a, 0, sizeof a);
  a.m8 = d_m;
  a.m_exp = d_m_exp;
  a.v8 = d_v;
  a.v_exp = d_v_exp;
  a.seed_lo = (uint32_t)seed;
  a.seed_hi = (uint32_t)(seed >> 32);
  const AdamCall c{n_tensors, n, w, grads, grad_dtype, copies, copy_dtype, state_elems, step,
                   lr, beta1, beta2, eps, weight_decay, d_grad_scale};
  return run_adamw(c, a, true, static_cast<hipStream_t>(stream));
}

int adamw_q8_values(const uint8_t* d_codes, const uint8_t* d_exp, int64_t elems, void* d_out,
                    int32_t out_dtype, emb_stream_t stream) {
  DENSE_CHECK(elems >= 0 && elems % EMB_ADAMW_BLOCK == 0, EMB_EINVAL,
              "adamw: elems must be a multiple of EMB_ADAMW_BLOCK");
  DENSE_CHECK(elems <= (int64_t)1 << 39, EMB_ERANGE, "adamw: more than 2^39 state elements");
  DENSE_CHECK(out_dtype == EMB_BF16 || out_dtype == EMB_F32, EMB_EINVAL,
              "adamw: values come in EMB_BF16 or EMB_F32");
  if (elems == 0) return EMB_OK;
  DENSE_CHECK(d_codes && d_exp && d_out, EMB_EINVAL, "adamw: null pointer");
  DENSE_CHECK(aligned(d_codes, 16) && aligned(d_out, 16), EMB_EINVAL,
              "adamw: codes or values not 16-byte aligned");
  return done(launch_adamw_values(d_codes, d_exp, elems, d_out, out_dtype,
                                  static_cast<hipStream_t>(stream)),
              "adamw_q8_values");
}

}  // extern "C"
