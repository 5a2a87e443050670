// Entry points of the paged cache (include/fg_attention.h): pages and slots of a
// step, rows into the cache, attention of one new token. Argument checks and
// launches; nothing is allocated or kept.
#include "fg_attention.h"
#include "fg_entry.hpp"
#include "fg_paged.hpp"
#include "fg_pages.hpp"

using namespace fg::ops;

namespace {

constexpr int64_t kMaxTokens = 0x7fffffff;

// The extent of a cache's tensor, `element` bytes each.
Rows extent(const void* p, int64_t element, int64_t pages, int64_t ps, int64_t rows, int64_t rs, int64_t heads, int64_t hs, int64_t dim) {
  return whole(p, element * ((pages - 1) * ps + (rows - 1) * rs + (heads - 1) * hs + dim));
}

// Do the caches of keys and values share memory? Ones of the same strides may lie within each other, as keys and values of a page, a token or a head do;
// others only if their pages do not.
bool caches_meet(const fg_append_t& k, const fg_append_t& v, int es, int64_t pages, int64_t page, int64_t heads, int64_t dim) {
  const bool same = (pages == 1 || k.page_stride == v.page_stride) && (page == 1 || k.row_stride == v.row_stride) && (heads == 1 || k.head_stride == v.head_stride);
  if (same) return meet({{pages, k.page_stride}, {page, k.row_stride}, {heads, k.head_stride}, {dim, 1}}, ((const char*)v.cache - (const char*)k.cache) / es);
  auto spans = [&](const fg_append_t& t) { return Rows{t.cache, pages, es * ((page - 1) * t.row_stride + (heads - 1) * t.head_stride + dim), es * t.page_stride}; };
  return overlap(spans(k), spans(v));
}

// Workgroups, two a compute unit: one round of its places for one head tile with 64 and 128 columns (3 and 2 fit) and two with 64 (2 fit). With 256
// columns, or 128 and more head tiles, registers leave one a compute unit, so that these take two rounds and twice the sums to join; the times
// below are with this target. Their work is equal. A workgroup may have a single unit of 128 tokens (4 requests of 300 tokens: two at least 8.4 us, one 6.3, and the join of twice
// the pieces 4.2 instead of 3.7).
constexpr int kPagedPlaces = 2 * kCUs;
int paged_target(int64_t parts) {
  const int64_t t = kPagedPlaces / parts;
  return (int)(t < 1 ? 1 : t);
}
// 16-head tiles of a workgroup, and the workgroups that this makes of all heads. More tiles read a cache fewer times, but a compute unit holds fewer
// waves with their sums; with neighbours on one die the second reader mostly finds the rows in its L2. 16 requests, one key head, bf16, us (e4m3
// caches follow the same rule, not measured by themselves):
//   dim, heads          16384 tokens each, 1, 2, 4 tiles      65536 tokens each
//   64, 32              22, 22                                58, 49
//   64, 64              33, 25, 39                            99, 61, 75
//   128, 32             31, 41                                110, 112
//   128, 64             47, 43, 64                            177, 143, 136
//   128, 128            81, 62, 62                            313, 238, 168
//   256, 32             63, 82                                224, 242
int head_tiles(int32_t group, int32_t dim) { return group <= 16 || dim == 256 ? 1 : dim == 64 ? 2 : group <= 32 ? 1 : group <= 64 ? 2 : 4; }
int64_t head_parts(int32_t kv, int32_t group, int32_t dim) {
  const int per = 16 * head_tiles(group, dim);
  return (int64_t)kv * ((group + per - 1) / per);
}

template <int D, bool E4M3>
void launch_paged(const PagedArgs& a, int tiles, dim3 grid, Launches& go) {
  const dim3 block(64 * kPagedWaves);
  if (tiles == 1) go(paged_kernel<D, E4M3, 1>, grid, block, 0, a);
  else if constexpr (D < 256) {
    if (tiles == 2) go(paged_kernel<D, E4M3, 2>, grid, block, 0, a);
    else if constexpr (D == 128) go(paged_kernel<D, E4M3, 4>, grid, block, 0, a);
  }
}

template <int D>
void launch_paged(bool e4m3, const PagedArgs& a, int tiles, dim3 grid, Launches& go) {
  e4m3 ? launch_paged<D, true>(a, tiles, grid, go) : launch_paged<D, false>(a, tiles, grid, go);
}

}  // namespace

extern "C" {

fg_status fg_page_step(const int32_t* lens, const int32_t* add, int32_t batch, int32_t* table, int64_t ldt, int32_t width,
                       int32_t* ring, const int64_t* ends, int32_t n_pages, int32_t page, int32_t* lens_out, int64_t* ends_out,
                       int32_t* starts, int64_t* slots, int32_t* positions, int32_t tokens, hipStream_t stream) {
  if (batch < 0 || width < 1 || n_pages < 1 || page < 1 || tokens < 0 || ldt < width || (int64_t)width * page > kMaxTokens) return FG_EINVAL;
  if (!starts || !ends || !ends_out || (batch && (!lens || !add || !table || !ring || !lens_out)) || (tokens && (!slots || !positions))) return FG_EINVAL;
  if (!aligned(lens, 4) || !aligned(add, 4) || !aligned(table, 4) || !aligned(ring, 4) || !aligned(ends, 8) || !aligned(lens_out, 4) ||
      !aligned(ends_out, 8) || !aligned(starts, 4) || !aligned(slots, 8) || !aligned(positions, 4))
    return FG_EINVAL;
  {
    const int64_t n = batch;
    const Rows l = whole(n ? lens : nullptr, 4 * n), d = whole(n ? add : nullptr, 4 * n), t{n ? table : nullptr, n, 4 * (int64_t)width, 4 * ldt};
    const Rows r = whole(ring, 4 * (int64_t)n_pages), e = whole(ends, 16), lo = whole(n ? lens_out : nullptr, 4 * n), eo = whole(ends_out, 16);
    const Rows st = whole(starts, 4 * (n + 1)), sl = whole(tokens ? slots : nullptr, 8 * (int64_t)tokens);
    const Rows po = whole(tokens ? positions : nullptr, 4 * (int64_t)tokens);
    if (overlaps(t, l, d, r, e, lo, eo, st, sl, po) || overlaps(r, l, d, e, lo, eo, st, sl, po) || overlaps(st, l, d, e, lo, eo, sl, po) ||
        overlaps(sl, l, d, e, lo, eo, po) || overlaps(po, l, d, e, lo, eo) || overlaps(lo, d, e, eo) || overlaps(eo, l, d) ||
        (lens_out != lens && overlap(lo, l)) || (ends_out != ends && overlap(eo, e)))
      return FG_EINVAL;
  }
  PageStepArgs a{lens, add, table, ring, ends, lens_out, ends_out, starts, slots, positions, ldt, batch, width, n_pages, page, tokens, 0};
  Launches go{stream};
  // few threads have shorter sums (64 requests: 256 threads 5.9 us, 1024 7.5); tokens by the one workgroup as long as each thread has a few, more by a
  // kernel of their own (64 requests, 4096 tokens 11.6 and 13.1 us, 8192 tokens 15.8 and 13.4)
  const bool few = batch <= 256 && tokens <= 1024;
  a.fill = few || tokens <= 4096;
  if (few) go(page_step_kernel<256>, dim3(1), dim3(256), 0, a);
  else go(page_step_kernel<1024>, dim3(1), dim3(1024), 0, a);
  if (!a.fill) {
    const int64_t n = ((int64_t)tokens + 1023) / 1024;
    go(page_slots_kernel, dim3((unsigned)(n < 8 * kCUs ? n : 8 * kCUs)), dim3(256), 0, a);
  }
  return go.status();
}

fg_status fg_kv_append(const fg_append_t* keys, const fg_append_t* values, int32_t cache_type, const int64_t* slots, int64_t rows,
                       int32_t heads, int32_t dim, int32_t n_pages, int32_t page, hipStream_t stream) {
  const bool e4m3 = cache_type == FG_E4M3;
  if (!keys || (!e4m3 && cache_type != FG_BF16) || rows < 0 || rows > 0x7fffffff || heads < 1 || heads > FG_ATTN_MAX_HEADS || dim < 8 || dim % 8 ||
      dim > FG_NORM_MAX_N || (e4m3 && dim > FG_APPEND_MAX_DIM) || n_pages < 1 || page < 1 || (int64_t)heads * dim > 0x7fffffff)
    return FG_EINVAL;
  if (rows == 0) return FG_OK;
  if (!slots || !aligned(slots, 8)) return FG_EINVAL;
  AppendArgs a{};
  a.slots = slots; a.rows = rows; a.n_slots = (int64_t)n_pages * page;
  a.heads = heads; a.dim = dim; a.page = page;
  const fg_append_t* part[2] = {keys, values};
  const int n = values ? 2 : 1, es = e4m3 ? 1 : 2;
  Rows in[2]{}, cache[2]{}, scale[2]{};
  for (int i = 0; i < n; ++i) {
    const fg_append_t& t = *part[i];
    if (!t.x || !t.cache || e4m3 != (t.scale != nullptr) || !aligned(t.x, 16) || !aligned(t.cache, 8 * es) || !aligned(t.scale, 4)) return FG_EINVAL;
    if (!multiple(t.x_row, 8) || !multiple(t.x_head, 8) || !multiple(t.page_stride, 8) || !multiple(t.row_stride, 8) || !multiple(t.head_stride, 8)) return FG_EINVAL;
    if (!distinct({{n_pages, t.page_stride}, {page, t.row_stride}, {heads, t.head_stride}, {dim, 1}})) return FG_EINVAL;
    a.x[i] = (const char*)t.x; a.cache[i] = (char*)t.cache; a.scale[i] = t.scale;
    a.x_row[i] = 2 * t.x_row; a.x_head[i] = 2 * t.x_head;
    a.c_page[i] = es * t.page_stride; a.c_tok[i] = es * t.row_stride; a.c_head[i] = es * t.head_stride;
    in[i] = rows3(t.x, 2, rows, t.x_row, heads, t.x_head, dim);
    cache[i] = extent(t.cache, es, n_pages, t.page_stride, page, t.row_stride, heads, t.head_stride, dim);
    scale[i] = whole(t.scale, 4 * a.n_slots * heads);
  }
  const Rows s = whole(slots, 8 * rows);
  for (int i = 0; i < n; ++i)
    if (overlaps(cache[i], s, in[0], in[1], scale[0], scale[1]) || overlaps(scale[i], s, in[0], in[1])) return FG_EINVAL;
  if (n == 2 && (overlap(scale[0], scale[1]) || caches_meet(*keys, *values, es, n_pages, page, heads, dim))) return FG_EINVAL;
  Launches go{stream};
  const int64_t pieces = e4m3 ? rows * heads * 16 : rows * heads * (dim / 8);
  if ((pieces + 255) / 256 > 0x7fffffff) return FG_EINVAL;
  dim3 grid = wide_grid((pieces + 255) / 256);
  grid.z = n;
  if (!e4m3) go(append_kernel, grid, dim3(256), 0, a);
  else if (dim <= 128) go(append8_kernel<1>, grid, dim3(256), 0, a);
  else if (dim <= 256) go(append8_kernel<2>, grid, dim3(256), 0, a);
  else go(append8_kernel<8>, grid, dim3(256), 0, a);
  return go.status();
}

fg_status fg_paged_attention_bytes(int32_t batch, int32_t kv, int32_t group, int32_t dim, int64_t* bytes) {
  if (!bytes || batch < 0 || batch > FG_ATTN_MAX_BATCH || kv < 1 || group < 1 || (int64_t)kv * group > FG_ATTN_MAX_HEADS ||
      (dim != 64 && dim != 128 && dim != 256))
    return FG_EINVAL;
  const int64_t items = batch + paged_target(head_parts(kv, group, dim)), rows = items * kv * group;
  *bytes = 4 * rows * dim + 8 * rows + 8 * (int64_t)batch;
  return FG_OK;
}

fg_status fg_paged_attention(const void* q, int64_t q_b, int64_t q_h, const fg_cache_t* k, const fg_cache_t* v, int32_t cache_type,
                             const fg_pages_t* pages, int32_t kv, int32_t group, int32_t dim, int32_t window, float scale,
                             void* workspace, int64_t workspace_bytes, void* out, int64_t out_b, int64_t out_h, float* lse,
                             int64_t lse_b, hipStream_t stream) {
  int64_t need = 0;
  const bool e4m3 = cache_type == FG_E4M3;
  if (!pages || !k || !v || (!e4m3 && cache_type != FG_BF16) || window < 0 || !(scale > 0.0f) || !(scale < __builtin_inff()) ||
      fg_paged_attention_bytes(pages->batch, kv, group, dim, &need) != FG_OK)
    return FG_EINVAL;
  if (pages->n_pages < 1 || pages->page < 16 || pages->page % 16 || pages->width < 1 || pages->ldt < pages->width ||
      (int64_t)pages->width * pages->page > kMaxTokens)
    return FG_EINVAL;
  const int64_t batch = pages->batch, heads = (int64_t)kv * group;
  // units of all requests are counted in 32 bits
  if (batch * ((int64_t)pages->width * pages->page / kPagedUnit + 2) > kMaxTokens) return FG_EINVAL;
  if (batch == 0) return FG_OK;
  if (!q || !k->data || !v->data || !pages->table || !pages->lens || !out || !workspace || workspace_bytes < need) return FG_EINVAL;
  if (e4m3 != (k->scale != nullptr) || e4m3 != (v->scale != nullptr)) return FG_EINVAL;
  if (!aligned(q, 16) || !aligned(k->data, 16) || !aligned(v->data, 16) || !aligned(k->scale, 16) || !aligned(v->scale, 16) || !aligned(out, 2) ||
      !aligned(lse, 4) || !aligned(workspace, 16) || !aligned(pages->table, 4) || !aligned(pages->lens, 4))
    return FG_EINVAL;
  const int es = e4m3 ? 1 : 2, step = 16 / es;
  for (const fg_cache_t* c : {k, v})
    if (!multiple(c->page_stride, step) || !multiple(c->row_stride, step) || !multiple(c->head_stride, step) || 16 * es * c->row_stride > kMaxTokens) return FG_EINVAL;
  if (!multiple(q_b, 8) || !multiple(q_h, 8) || out_b < 0 || out_h < 0 || (lse && lse_b < heads && batch > 1)) return FG_EINVAL;
  if (!distinct({{batch, out_b}, {heads, out_h}, {dim, 1}})) return FG_EINVAL;
  const int64_t p = pages->page, n = pages->n_pages;
  const Rows ws = whole(workspace, need), o = rows3(out, 2, batch, out_b, heads, out_h, dim), qr = rows3(q, 2, batch, q_b, heads, q_h, dim);
  const Rows kr = extent(k->data, es, n, k->page_stride, p, k->row_stride, kv, k->head_stride, dim);
  const Rows vr = extent(v->data, es, n, v->page_stride, p, v->row_stride, kv, v->head_stride, dim);
  const Rows ks = whole(k->scale, 4 * n * kv * p), vs = whole(v->scale, 4 * n * kv * p), le = whole(pages->lens, 4 * batch);
  const Rows t{pages->table, batch, 4 * (int64_t)pages->width, 4 * pages->ldt}, ls{lse, batch, 4 * heads, 4 * lse_b};
  if (overlaps(o, qr, kr, vr, ks, vs, t, le, ws, ls) || overlaps(ls, qr, kr, vr, ks, vs, t, le, ws) || overlaps(ws, qr, kr, vr, ks, vs, t, le))
    return FG_EINVAL;
  PagedArgs a{};
  const int64_t parts = head_parts(kv, group, dim);
  const int target = paged_target(parts);
  const int64_t items = batch + target;
  char* w = (char*)workspace;
  a.part = (float*)w;
  a.ml = (float*)(w + 4 * items * heads * dim);
  a.split = SplitArgs{pages->lens, pages->table, pages->ldt, pages->batch, pages->width, pages->n_pages, pages->page, window, target,
                      (int32_t*)(w + (4 * dim + 8) * items * heads)};
  a.q = (const char*)q; a.k = (const char*)k->data; a.v = (const char*)v->data; a.ks = k->scale; a.vs = v->scale;
  a.out = (uint16_t*)out; a.lse = lse;
  a.q_b = 2 * q_b; a.q_h = 2 * q_h; a.out_b = out_b; a.out_h = out_h; a.lse_b = lse_b;
  a.k_page = es * k->page_stride; a.k_head = es * k->head_stride; a.k_tok = (int32_t)(es * k->row_stride);
  a.v_page = es * v->page_stride; a.v_head = es * v->head_stride; a.v_tok = (int32_t)(es * v->row_stride);
  a.kv = kv; a.group = group; a.heads = (int32_t)heads; a.c = scale * kLog2E;
  Launches go{stream};
  const dim3 grid((unsigned)((target + 7) / 8 * 8 * parts));
  const int tiles = head_tiles(group, dim);
  if (dim == 64) launch_paged<64>(e4m3, a, tiles, grid, go);
  else if (dim == 128) launch_paged<128>(e4m3, a, tiles, grid, go);
  else launch_paged<256>(e4m3, a, tiles, grid, go);
  // a table this narrow leaves one unit, and so one piece, a request
  if ((int64_t)pages->width * pages->page > kPagedUnit) {
    const JoinArgs j{a.split.pieces, a.part, a.ml, a.out, lse, out_b, out_h, lse_b, (int32_t)heads};
    if (dim == 64) launch_join<64>(j, batch, target, go);
    else if (dim == 128) launch_join<128>(j, batch, target, go);
    else launch_join<256>(j, batch, target, go);
  }
  return go.status();
}

}  // extern "C"
