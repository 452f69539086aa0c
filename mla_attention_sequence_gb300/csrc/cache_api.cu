// C ABI of the norms with rotation and of the paged 4-bit latent cache. Argument checks, workspace
// layout, dispatch.
#include "api_util.h"
#include "cache4.h"

#include <algorithm>
#include <cmath>

namespace laga {
namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

laga_status check_eps(float eps) {
  // below, the smallest rows' squares and eps both leave fp32; above, its square does
  if (!(eps >= 1e-30f && eps <= 1e10f)) return fail(LAGA_ERR_INVALID_ARG, "eps must be between 1e-30 and 1e10%s");
  return LAGA_OK;
}

// The descriptor's checks that norm_rope and its backward share.
laga_status norm_plan(const laga_mla_rope_desc* desc, float eps, const void* pos, const void* q, const void* k_rope,
                      const void* w_q, const void* w_k, NormArgs* a, const RopeTable** t) {
  laga_status st = rope_plan(desc, pos, &a->rope, t);
  if (st == LAGA_OK) st = check_eps(eps);
  if (st != LAGA_OK) return st;
  if (a->rope.inverse) return fail(LAGA_ERR_INVALID_ARG, "norm_rope: the rotation comes after the norm (no inverse)%s");
  if (a->rope.d_nope + a->rope.d_rope > kNormWidth)
    return fail(LAGA_ERR_UNSUPPORTED, "norm_rope: d_nope + d_rope <= 1024%s");
  if ((!q && !k_rope) || !q != !w_q || !k_rope != !w_k)
    return fail(LAGA_ERR_INVALID_ARG, "norm_rope: q or k_rope, each with its weight%s");
  a->eps = eps;
  a->rope.q = q;
  a->rope.k = k_rope;
  a->w_q = w_q;
  a->w_k = w_k;
  return LAGA_OK;
}

laga_status check_cache(const laga_mla_cache4* c, CacheView* v, bool sizes_only) {
  if (!c) return fail(LAGA_ERR_INVALID_ARG, "null cache%s");
  if (c->dtype != LAGA_DTYPE_F32 && c->dtype != LAGA_DTYPE_BF16)
    return fail(LAGA_ERR_UNSUPPORTED, "dtype must be LAGA_DTYPE_F32 or LAGA_DTYPE_BF16%s");
  if (c->pages < 1 || c->page_size < 1 || c->d_c < 1 || c->d_rope < 0)
    return fail(LAGA_ERR_INVALID_ARG, "cache: pages, page_size, d_c >= 1, d_rope >= 0%s");
  if (c->pages >= (int64_t(1) << 31) || c->page_size > 65536 || c->d_c > 1024 || c->d_rope > 256)
    return fail(LAGA_ERR_UNSUPPORTED, "cache: page_size <= 65536, d_c <= 1024, d_rope <= 256%s");
  if (!sizes_only) {
    if (!c->codes || !c->scales || !aligned16(c->codes) || !aligned16(c->scales))
      return fail(LAGA_ERR_INVALID_ARG, "cache: codes and scales must be non-null and 16-byte aligned%s");
    if (c->d_rope > 0 && (!c->k_rope || !aligned16(c->k_rope)))
      return fail(LAGA_ERR_INVALID_ARG, "cache: k_rope must be non-null and 16-byte aligned%s");
  }
  v->codes = c->codes;
  v->scales = c->scales;
  v->keys = c->k_rope;
  v->pages = c->pages;
  v->page = static_cast<int>(c->page_size);
  v->d_c = static_cast<int>(c->d_c);
  v->d_rope = static_cast<int>(c->d_rope);
  v->is_bf16 = c->dtype == LAGA_DTYPE_BF16;
  return LAGA_OK;
}

laga_status check_rows(int64_t batch, int64_t rows, int64_t max_pages, const int32_t* table, const int32_t* starts,
                       const int32_t* counts, CacheRows* r) {
  if (batch < 1 || rows < 1 || max_pages < 1)
    return fail(LAGA_ERR_INVALID_ARG, "cache rows: batch, rows, max_pages >= 1%s");
  if (batch >= (int64_t(1) << 31) || rows >= (int64_t(1) << 31) || batch * rows >= (int64_t(1) << 31) ||
      max_pages >= (int64_t(1) << 31))
    return fail(LAGA_ERR_UNSUPPORTED, "problem too large%s");
  if (!table || !starts || !aligned_to(table, 4) || !aligned_to(starts, 4) || !aligned_to(counts, 4))
    return fail(LAGA_ERR_INVALID_ARG, "table and starts must be non-null, and they and counts 4-byte aligned%s");
  r->pages = PageTable{table, static_cast<int>(batch), static_cast<int>(max_pages)};
  r->rows = static_cast<int>(rows);
  r->starts = starts;
  r->counts = counts;
  return LAGA_OK;
}

// Which form of the tensor cores: mma.sync's time goes with the tiles of 16 rows, the tcgen05 form's with
// tiles of 128, and it begins later. Kernel's time in us at 16, 32, 48 and 64 rows a sequence, mma.sync :
// tcgen05 (events):
//   48 sequences of 2000 .. 8192 tokens   55 : 94    94 : 89    133 : 90    174 : 88
//   8 of them                             20 : 29    27 : 30    35 : 29     41 : 30
//   4 of 500 .. 2000                      12 : 16    14 : 14    16 : 15     18 : 14
//   one of 8000                           14 : 19    16 : 18    17 : 18     19 : 17
//   one of 600                            10 : 14    10 : 14    11 : 14     12 : 14
// So mma.sync up to 32 rows, and up to 64 while what the table has room for is at most about three of its
// key tiles for each of its CTAs. The lengths are on the GPU, so the table's width stands for them: in a table
// far wider than its sequences 33 to 64 rows take the tcgen05 form (one of 600: 14 us for 11), whose bits differ.
constexpr int kFewRows = 32, kFewRowsShort = 64, kShortTiles = 3;

struct AttnSizes {
  CacheAttn a;
  int d_nope, d_v;
  bool tc, few;  // tensor cores; mma.sync's form of them
  size_t items_bytes, parts_bytes, hull_bytes, query_bytes, up_bytes, ctx_bytes, ml_bytes, o_bytes;
  size_t total() const {
    return items_bytes + parts_bytes + hull_bytes + query_bytes + up_bytes + ctx_bytes + ml_bytes + o_bytes;
  }
};

laga_status attn_plan(const laga_mla_cache4_desc* d, const laga_mla_cache4* cache, bool sizes_only, AttnSizes* s) {
  if (!d) return fail(LAGA_ERR_INVALID_ARG, "null descriptor%s");
  CacheAttn& a = s->a;
  a = CacheAttn{};
  const laga_status st = check_cache(cache, &a.cache, sizes_only);
  if (st != LAGA_OK) return st;
  if (d->batch < 1 || d->sq < 1 || d->n_h < 1 || d->max_pages < 1 || d->d_nope < 1 || d->d_v < 1)
    return fail(LAGA_ERR_INVALID_ARG, "cache attention: batch, sq, n_h, max_pages, d_nope, d_v >= 1%s");
  if (d->variant != LAGA_VARIANT_AUTO && d->variant != LAGA_VARIANT_SIMT)
    return fail(LAGA_ERR_UNSUPPORTED, "cache attention: variants AUTO and SIMT%s");
  if (d->d_nope + cache->d_rope > 256 || d->d_v > 256)
    return fail(LAGA_ERR_UNSUPPORTED, "cache attention: d_nope + d_rope <= 256 and d_v <= 256%s");
  const int64_t lim = int64_t(1) << 31;
  if (d->batch >= lim || d->sq >= lim || d->n_h >= 65536 || d->max_pages >= lim || d->batch * d->sq >= lim / 2 ||
      d->batch * d->sq * d->n_h >= lim)
    return fail(LAGA_ERR_UNSUPPORTED, "problem too large%s");
  if (std::isnan(d->softmax_scale) || std::isinf(d->softmax_scale))
    return fail(LAGA_ERR_INVALID_ARG, "softmax_scale must be finite%s");
  a.pages = PageTable{nullptr, static_cast<int>(d->batch), static_cast<int>(d->max_pages)};
  a.Sq = static_cast<int>(d->sq);
  a.n_h = static_cast<int>(d->n_h);
  if (d->sq * d->n_h >= lim) return fail(LAGA_ERR_UNSUPPORTED, "problem too large%s");
  a.rows = a.Sq * a.n_h;
  a.causal = d->causal != 0;
  s->d_nope = static_cast<int>(d->d_nope);
  s->d_v = static_cast<int>(d->d_v);
  a.scale = d->softmax_scale > 0.f ? d->softmax_scale
                                   : 1.f / std::sqrt(static_cast<float>(d->d_nope + cache->d_rope));
  s->tc = d->variant == LAGA_VARIANT_AUTO && a.cache.is_bf16 && a.cache.d_c == 512 && a.cache.d_rope == 64 &&
          s->d_nope == 128 && s->d_v == 128;
  const double short_tiles = static_cast<double>(d->batch) * ((a.rows + kMmaRows - 1) / kMmaRows) * d->max_pages * cache->page_size / kMmaKeys;
  s->few = s->tc && (a.rows <= kFewRows || (a.rows <= kFewRowsShort && short_tiles <= kShortTiles * 2. * sm_count()));
  a.tile = s->few ? kMmaRows : s->tc ? kTcRows : kSimtRows;
  a.keys = s->few ? kMmaKeys : s->tc ? kTcKeys : kSimtKeys;
  // tcgen05: two CTAs a part, one a SM; else one, two a SM
  a.parts = s->tc && !s->few ? sm_count() / 2 : 2 * sm_count();
  a.row_tiles = (a.rows + a.tile - 1) / a.tile;
  const int64_t items = static_cast<int64_t>(a.pages.B) * a.row_tiles;
  const int64_t room = std::min(d->max_pages * cache->page_size, lim - 1);
  if (items * (room / a.keys + 2) >= lim || room > lim - 2 * a.keys)
    return fail(LAGA_ERR_UNSUPPORTED, "cache attention: problem too large (rows times the table's room)%s");
  s->items_bytes = align_up((items + 1) * sizeof(int), 256);
  s->parts_bytes = align_up(a.parts * sizeof(int), 256);
  s->hull_bytes = align_up(items * sizeof(int2), 256);
  const size_t rows = static_cast<size_t>(a.pages.B) * a.rows;
  s->ctx_bytes = align_up(rows * a.cache.d_c * 4, 256);
  s->query_bytes = s->tc ? align_up(rows * kQueryBytes, 256) : s->ctx_bytes;  // CUDA cores: q_lat in fp32
  s->up_bytes = s->tc ? align_up(rows * 4, 256) : 0;
  s->ml_bytes = align_up(static_cast<size_t>(2) * a.parts * a.tile * sizeof(float2), 256);
  s->o_bytes = align_up(static_cast<size_t>(2) * a.parts * a.tile * a.cache.d_c * 4, 256);
  return LAGA_OK;
}

}  // namespace
}  // namespace laga

using namespace laga;

extern "C" {

laga_status laga_mla_norm_rope(const laga_mla_rope_desc* desc, float eps, const void* pos, const void* q,
                               const void* k_rope, const void* q_weight, const void* k_weight, void* q_out, void* k_out,
                               laga_stream_t stream) {
  NormArgs a{};
  const RopeTable* t = nullptr;
  const laga_status st = norm_plan(desc, eps, pos, q, k_rope, q_weight, k_weight, &a, &t);
  if (st != LAGA_OK) return st;
  if (!q != !q_out || !k_rope != !k_out)
    return fail(LAGA_ERR_INVALID_ARG, "norm_rope: q or k_rope, each with its output%s");
  const uintptr_t e = a.rope.is_bf16 ? 2 : 4;
  for (const void* p : {q, k_rope, q_weight, k_weight, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    if (!aligned_to(p, e)) return fail(LAGA_ERR_INVALID_ARG, "norm_rope: tensors must be aligned to their type%s");
  a.rope.q_out = q_out;
  a.rope.k_out = k_out;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_launch(timed("norm_rope", s, [&] { return norm_rope(a, *t, s); }));
}

size_t laga_mla_norm_rope_bwd_workspace_size(const laga_mla_rope_desc* desc) {
  RopeArgs a{};
  const RopeTable* t = nullptr;
  if (rope_plan(desc, desc, &a, &t) != LAGA_OK || a.d_nope + a.d_rope > kNormWidth) return 0;
  return align_up(norm_rope_bwd_partials(a) * sizeof(float), 256);
}

laga_status laga_mla_norm_rope_bwd(const laga_mla_rope_desc* desc, float eps, const void* pos, const void* dq_out,
                                   const void* dk_out, const void* q, const void* k_rope, const void* q_weight,
                                   const void* k_weight, void* dq, void* dk_rope, void* dq_weight, void* dk_weight,
                                   void* workspace, size_t workspace_bytes, laga_stream_t stream) {
  NormArgs a{};
  const RopeTable* t = nullptr;
  const laga_status st = norm_plan(desc, eps, pos, q, k_rope, q_weight, k_weight, &a, &t);
  if (st != LAGA_OK) return st;
  if (!q != !dq_out || !q != !dq || !q != !dq_weight || !k_rope != !dk_out || !k_rope != !dk_rope || !k_rope != !dk_weight)
    return fail(LAGA_ERR_INVALID_ARG, "norm_rope_bwd: q or k_rope, each with its gradients%s");
  const uintptr_t e = a.rope.is_bf16 ? 2 : 4;
  for (const void* p : {q, k_rope, q_weight, k_weight, dq_out, dk_out, static_cast<const void*>(dq),
                        static_cast<const void*>(dk_rope), static_cast<const void*>(dq_weight),
                        static_cast<const void*>(dk_weight)})
    if (!aligned_to(p, e)) return fail(LAGA_ERR_INVALID_ARG, "norm_rope_bwd: tensors must be aligned to their type%s");
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < norm_rope_bwd_partials(a.rope) * sizeof(float))
    return fail(LAGA_ERR_WORKSPACE, "workspace missing, misaligned (256 B) or too small%s");
  a.z_q = dq_out;
  a.z_k = dk_out;
  a.rope.q_out = dq;
  a.rope.k_out = dk_rope;
  a.dw_q = dq_weight;
  a.dw_k = dk_weight;
  a.partials = static_cast<float*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_launch(timed("norm_rope_bwd", s, [&] { return norm_rope_bwd(a, *t, s); }));
}

laga_status laga_mla_cache4_append(const laga_mla_cache4* cache, int64_t batch, int64_t rows, int64_t max_pages,
                                   const int32_t* table, const int32_t* starts, const int32_t* counts, const void* c_kv,
                                   const void* k_rope, const void* k_weight, float eps, const laga_mla_rope_desc* rope,
                                   const void* pos, laga_stream_t stream) {
  CacheAppend a{};
  laga_status st = check_cache(cache, &a.cache, false);
  if (st == LAGA_OK) st = check_rows(batch, rows, max_pages, table, starts, counts, &a.at);
  if (st != LAGA_OK) return st;
  const uintptr_t e = a.cache.is_bf16 ? 2 : 4;
  if (!c_kv || (a.cache.d_rope > 0 && !k_rope) || !aligned_to(c_kv, e) || !aligned_to(k_rope, e) || !aligned_to(k_weight, e))
    return fail(LAGA_ERR_INVALID_ARG, "cache4_append: c_kv and k_rope must be non-null, all aligned to their type%s");
  if (k_weight && (st = check_eps(eps)) != LAGA_OK) return st;
  static const RopeTable none{};
  const RopeTable* t = &none;
  a.turn = rope != nullptr && a.cache.d_rope > 0;
  if (a.turn) {
    a.own_pos = pos != nullptr;
    laga_mla_rope_desc x = *rope;  // the rows have no heads, and without pos no type of it
    x.n_h = 1;
    x.d_nope = 0;
    if (!pos) x.pos64 = 0;
    st = rope_plan(&x, pos ? pos : starts, &a.rope, &t);
    if (st != LAGA_OK) return st;
    if (rope->d_rope != cache->d_rope || rope->tokens != batch * rows || rope->dtype != cache->dtype || rope->inverse)
      return fail(LAGA_ERR_INVALID_ARG, "cache4_append: the rotation's tokens, d_rope and dtype are the rows' and the cache's, not inverse%s");
    if (!pos && rope->n_axes != 1)
      return fail(LAGA_ERR_INVALID_ARG, "cache4_append: rows turned by their positions in the cache have one axis%s");
  }
  a.c_kv = c_kv;
  a.k_rope = k_rope;
  a.w_k = k_weight;
  a.eps = eps;
  a.status = device_status_ptr();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_launch(timed("cache4_append", s, [&] { return cache4_append(a, *t, s); }));
}

laga_status laga_mla_cache4_read(const laga_mla_cache4* cache, int64_t batch, int64_t rows, int64_t max_pages,
                                 const int32_t* table, const int32_t* starts, const int32_t* counts, void* c_kv,
                                 void* k_rope, laga_stream_t stream) {
  CacheRead a{};
  laga_status st = check_cache(cache, &a.cache, false);
  if (st == LAGA_OK) st = check_rows(batch, rows, max_pages, table, starts, counts, &a.at);
  if (st != LAGA_OK) return st;
  const uintptr_t e = a.cache.is_bf16 ? 2 : 4;
  if (!c_kv || (a.cache.d_rope > 0 && !k_rope) || !aligned_to(c_kv, e) || !aligned_to(k_rope, e))
    return fail(LAGA_ERR_INVALID_ARG, "cache4_read: c_kv and k_rope must be non-null and aligned to their type%s");
  a.c_kv = c_kv;
  a.k_rope = k_rope;
  a.status = device_status_ptr();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return from_launch(timed("cache4_read", s, [&] { return cache4_read(a, s); }));
}

size_t laga_mla_cache4_fwd_workspace_size(const laga_mla_cache4_desc* desc, const laga_mla_cache4* cache) {
  AttnSizes s{};
  return attn_plan(desc, cache, true, &s) == LAGA_OK ? s.total() : 0;
}

laga_status laga_mla_cache4_fwd(const laga_mla_cache4_desc* desc, const laga_mla_cache4* cache, const laga_mla_mods* mods,
                                const int32_t* table, const int32_t* lengths, const void* q, const void* W_UK,
                                const void* W_UV, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                laga_stream_t stream) {
  AttnSizes z{};
  laga_status st = attn_plan(desc, cache, false, &z);
  if (st != LAGA_OK) return st;
  CacheAttn& a = z.a;
  st = check_mods(mods, &a.mods);
  if (st != LAGA_OK) return st;
  for (const void* p : {q, W_UK, W_UV, static_cast<const void*>(out), static_cast<const void*>(lse)})
    if (!p || !aligned16(p)) return fail(LAGA_ERR_INVALID_ARG, "tensor pointers must be non-null and 16-byte aligned%s");
  if (!table || !lengths || !aligned_to(table, 4) || !aligned_to(lengths, 4))
    return fail(LAGA_ERR_INVALID_ARG, "table and lengths must be non-null and 4-byte aligned%s");
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < z.total())
    return fail(LAGA_ERR_WORKSPACE, "workspace missing, misaligned (256 B) or too small%s");
  a.pages.table = table;
  a.lengths = lengths;
  a.key_lo = mods ? mods->key_lo : nullptr;
  a.key_hi = mods ? mods->key_hi : nullptr;
  a.lse = lse;
  a.status = device_status_ptr();
  char* at = static_cast<char*>(workspace);
  auto take = [&](size_t n) {
    char* p = at;
    at += n;
    return p;
  };
  a.first = reinterpret_cast<int*>(take(z.items_bytes));
  a.part_item = reinterpret_cast<int*>(take(z.parts_bytes));
  a.hull = reinterpret_cast<int2*>(take(z.hull_bytes));
  CacheOperands x;
  x.query = reinterpret_cast<uint8_t*>(take(z.query_bytes));
  x.up = reinterpret_cast<float*>(take(z.up_bytes));
  x.ctx = reinterpret_cast<float*>(take(z.ctx_bytes));
  a.part_ml = reinterpret_cast<float2*>(take(z.ml_bytes));
  a.part_o = reinterpret_cast<float*>(take(z.o_bytes));
  const bool b16 = a.cache.is_bf16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  LaunchResult r;
  if (z.tc) {
    auto cb = [](const void* p) { return static_cast<const bf16*>(p); };
    r = timed("cache4_prepare", s, [&] { return cache4_tc_prepare(a, cb(q), cb(W_UK), x, s); });
    if (r.ok()) r = timed("cache4_attn", s, [&] { return z.few ? cache4_mma_attn(a, x, s) : cache4_tc_attn(a, x, s); });
    if (r.ok()) r = timed("cache4_finish", s, [&] { return cache4_tc_finish(a, x, cb(W_UV), static_cast<bf16*>(out), s); });
    return from_launch(r);
  }
  float* q_lat = reinterpret_cast<float*>(x.query);
  r = timed("cache4_prepare", s, [&] { return cache4_simt_prepare(a, b16, z.d_nope, q, W_UK, q_lat, s); });
  if (r.ok()) r = timed("cache4_attn", s, [&] { return cache4_simt_attn(a, b16, z.d_nope, q, q_lat, x.ctx, s); });
  if (r.ok()) r = timed("cache4_join", s, [&] { return cache4_join(a, x.ctx, s); });
  if (r.ok()) r = timed("cache4_out", s, [&] { return cache4_simt_out(a, b16, z.d_v, x.ctx, W_UV, out, s); });
  return from_launch(r);
}

}  // extern "C"
