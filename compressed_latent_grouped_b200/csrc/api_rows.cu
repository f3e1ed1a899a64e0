// C ABI of the operators on finished query / key / value rows: the append with
// the rotation and the cache read-back.  Host-side validation and dispatch, as
// in api.cu: nothing is launched on a bad argument.
#include <algorithm>

#include "api_internal.h"

namespace ccgqa {
namespace {

// A tensor [n0, n1, n2, d] of head rows: aligned, and no two rows share memory.
bool rows_ok(const Geo& g, const ccgqa_rows& r, int64_t batch, int64_t tokens, int64_t heads) {
  if (!r.ptr || !aligned16(r.ptr)) return false;
  struct Dim {
    int64_t stride, n;
  } d[3] = {{r.batch, batch}, {r.token, tokens}, {r.head, heads}};
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  constexpr int64_t kMax = int64_t(1) << 39;   // keeps every product below in range
  int64_t extent = g.d;
  for (const Dim& x : d) {
    if (x.n <= 1) continue;
    if (x.stride < extent || x.stride > kMax || (x.stride * static_cast<int64_t>(g.es)) % 16 != 0)
      return false;
    if (x.n > kMax / x.stride) return false;
    extent += (x.n - 1) * x.stride;
  }
  return true;
}
Rows rows_of(const ccgqa_rows& r, int64_t batch, int64_t tokens, int64_t heads) {
  // the stride of a dimension of one is never used; zero keeps it out of the arithmetic
  return Rows{r.ptr, batch > 1 ? r.batch : 0, tokens > 1 ? r.token : 0, heads > 1 ? r.head : 0};
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// Validate the 8-bit description of a cache (null: the working type).
ccgqa_status check_cache8(const ccgqa_kvcache* c, const ccgqa_cache8* c8) {
  if (!c8) return CCGQA_OK;
  if (c8->format != CCGQA_CACHE_I8 && c8->format != CCGQA_CACHE_E4M3) return CCGQA_ERR_INVALID_ARG;
  const int b = c8->block;
  if (b != 16 && b != 32 && b != 64 && b != 128) return CCGQA_ERR_INVALID_ARG;
  if (c->cap % b != 0 || (c->block_table && b > c->page_size)) return CCGQA_ERR_INVALID_ARG;
  if (!c8->k_scale || !c8->v_scale || (reinterpret_cast<uintptr_t>(c8->k_scale) & 3) ||
      (reinterpret_cast<uintptr_t>(c8->v_scale) & 3))
    return CCGQA_ERR_INVALID_ARG;
  return CCGQA_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

template <typename T>
cudaError_t run_append(const Geo& g, const ccgqa_kvcache* c, const ccgqa_cache8* c8,
                       const ccgqa_append* a, int32_t* dev_err, cudaStream_t st) {
  AppendArgs<T> x{};
  x.ck = c->k;
  x.cv = c->v;
  if (c8) {
    x.k_scale = c8->k_scale;
    x.v_scale = c8->v_scale;
    x.block_shift = log2_of(c8->block);
  }
  x.pages = page_map(c);
  x.len = c->len;
  x.cap = c->cap;
  x.B = c->batch;
  x.Hq = g.Hq;
  x.Hkv = g.Hkv;
  x.d = g.d;
  x.n_new = a->n_new;
  auto rows = [&](const ccgqa_rows& r, int heads) { return rows_of(r, x.B, x.n_new, heads); };
  x.q = rows(a->q, g.Hq);
  x.q_out = rows(a->q_out, g.Hq);
  x.k = rows(a->k, g.Hkv);
  x.v = rows(a->v, g.Hkv);
  x.k_out = rows(a->k_out, g.Hkv);
  x.n_valid = a->n_valid;
  x.pos = a->pos;
  x.rope_on = g.rope_on;
  if (g.rope_on)
    for (int i = 0; i < g.d / 2; ++i) x.rope_frac[i] = rope_turn_fraction(g.rope_log2_base, i, g.d);
  x.dev_err = dev_err;
  return launch_append_rope<T>(x, c8 ? c8->format : 0, st);
}

}  // namespace
}  // namespace ccgqa

using namespace ccgqa;

CCGQA_API ccgqa_status ccgqa_kvcache_append_rope(const ccgqa_config* cfg,
                                                 const ccgqa_kvcache* cache,
                                                 const ccgqa_cache8* c8, const ccgqa_append* a,
                                                 int32_t* dev_err, void* stream) {
  Geo g;
  ccgqa_status s = derive(cfg, &g);
  if (s != CCGQA_OK) return s;
  if ((s = check_cache(g, cache, false)) != CCGQA_OK) return s;
  if ((s = check_cache8(cache, c8)) != CCGQA_OK) return s;
  if (!a || a->n_new < 0) return CCGQA_ERR_INVALID_ARG;
  if (a->n_new > cache->cap) return CCGQA_ERR_CAPACITY;
  if (a->n_new == 0) return CCGQA_OK;
  const int64_t B = cache->batch, n = a->n_new;
  if (!rows_ok(g, a->k, B, n, g.Hkv) || !rows_ok(g, a->v, B, n, g.Hkv)) return CCGQA_ERR_INVALID_ARG;
  if ((a->q.ptr == nullptr) != (a->q_out.ptr == nullptr)) return CCGQA_ERR_INVALID_ARG;
  if (a->q.ptr && (!rows_ok(g, a->q, B, n, g.Hq) || !rows_ok(g, a->q_out, B, n, g.Hq)))
    return CCGQA_ERR_INVALID_ARG;
  if (a->k_out.ptr && !rows_ok(g, a->k_out, B, n, g.Hkv)) return CCGQA_ERR_INVALID_ARG;
  if (!aligned4(a->n_valid) || !aligned4(a->pos)) return CCGQA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!stream_allowed(st)) return CCGQA_ERR_INVALID_ARG;
  const cudaError_t e = g.dtype == CCGQA_BF16 ? run_append<bf16>(g, cache, c8, a, dev_err, st)
                                              : run_append<float>(g, cache, c8, a, dev_err, st);
  return e == cudaSuccess ? CCGQA_OK : cuda_fail(e);
}

CCGQA_API ccgqa_status ccgqa_kvcache_read(const ccgqa_config* cfg, const ccgqa_kvcache* cache,
                                          const ccgqa_cache8* c8, int32_t first, int32_t n,
                                          const ccgqa_rows* k_out, const ccgqa_rows* v_out,
                                          int32_t* dev_err, void* stream) {
  Geo g;
  ccgqa_status s = derive(cfg, &g);
  if (s != CCGQA_OK) return s;
  if ((s = check_cache(g, cache, false)) != CCGQA_OK) return s;
  if ((s = check_cache8(cache, c8)) != CCGQA_OK) return s;
  if (first < 0 || n < 0) return CCGQA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(first) + n > cache->cap) return CCGQA_ERR_CAPACITY;
  if (n == 0) return CCGQA_OK;
  if (!k_out || !v_out || !rows_ok(g, *k_out, cache->batch, n, g.Hkv) ||
      !rows_ok(g, *v_out, cache->batch, n, g.Hkv))
    return CCGQA_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!stream_allowed(st)) return CCGQA_ERR_INVALID_ARG;
  ReadArgs a{};
  a.ck = cache->k;
  a.cv = cache->v;
  if (c8) {
    a.k_scale = c8->k_scale;
    a.v_scale = c8->v_scale;
    a.block_shift = log2_of(c8->block);
  }
  a.pages = page_map(cache);
  a.len = cache->len;
  a.cap = cache->cap;
  a.B = cache->batch;
  a.Hkv = g.Hkv;
  a.d = g.d;
  a.first = first;
  a.n = n;
  a.k_out = rows_of(*k_out, cache->batch, n, g.Hkv);
  a.v_out = rows_of(*v_out, cache->batch, n, g.Hkv);
  a.dev_err = dev_err;
  const int fmt = c8 ? c8->format : 0;
  const cudaError_t e =
      g.dtype == CCGQA_BF16 ? launch_kv_read<bf16>(a, fmt, st) : launch_kv_read<float>(a, fmt, st);
  return e == cudaSuccess ? CCGQA_OK : cuda_fail(e);
}
