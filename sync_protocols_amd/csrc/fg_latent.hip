// Entry points of latent attention (include/fg_attention.h): the absorbed form of one
// new token over a paged cache, and the expanded form of prompts.
#include "fg_attention.h"
#include "fg_entry.hpp"
#include "fg_latent.hpp"
#include "fg_prompt.hpp"

using namespace fg::ops;

namespace {

constexpr int64_t kMax = 0x7fffffff;

bool sizes_ok(int32_t heads, int32_t rank, int32_t rope, int32_t nope, float scale) {
  return heads >= 1 && heads <= FG_ATTN_MAX_HEADS && (rank == 256 || rank == 512) && (rope == 32 || rope == 64) && (nope == 64 || nope == 128) &&
         scale > 0.0f && scale < __builtin_inff();
}

// 16-head tiles of a workgroup, and the workgroups that this makes of all heads.
int head_tiles(int32_t heads) { return heads <= 16 ? 1 : heads <= 32 ? 2 : 4; }
// Absorbed queries, twice where they are pairs.
int64_t query_bytes(int64_t batch, int32_t heads, int32_t row) { return batch * heads * row * (heads <= 16 ? 4 : 2); }
int64_t head_parts(int32_t heads) { return (heads + 16 * head_tiles(heads) - 1) / (16 * head_tiles(heads)); }
// Workgroups of four waves that share tiles of 64 rows, one a compute unit, or, up to 32 heads, of two waves and 32 rows, two a unit: their LDS fills it with rank
// 512, their registers with rank 256 and two head tiles. With one head tile of rank 256 three would fit; two are taken all the same.
int latent_tile(int32_t heads) { return head_tiles(heads) > 2 ? 64 : 32; }
int latent_target(int32_t heads) {
  const int64_t t = kCUs * (64 / latent_tile(heads)) / head_parts(heads);
  return (int)(t < 1 ? 1 : t);
}

template <int R, int P, int G, int HW>
void launch_latent(const LatentArgs& a, dim3 grid, Launches& go) {
  go(latent_kernel<R, P, G, HW>, grid, dim3(128 * G), LatentShape<R, P, G, HW>::LDS, a);
}
template <int R, int P>
void launch_latent(const LatentArgs& a, dim3 grid, Launches& go) {
  switch (head_tiles(a.heads)) {
    case 1: launch_latent<R, P, 1, 1>(a, grid, go); break;
    case 2: launch_latent<R, P, 1, 2>(a, grid, go); break;
    default: launch_latent<R, P, 2, 2>(a, grid, go);
  }
}

// Many pieces a request: more than 16, if lengths are even.
template <int R, bool MANY>
void launch_join_as(const LatentArgs& a, Launches& go) {
  typedef LatentJoinShape<R, MANY> Sh;
  go(latent_join_kernel<R, MANY>, dim3((unsigned)a.tiles, (unsigned)a.split.batch, Sh::Z), dim3(64 * Sh::WAVES), 0, a);
}
template <int R>
void launch_join(const LatentArgs& a, Launches& go) {
  const bool many = a.split.target > 16 * a.split.batch;
  many ? launch_join_as<R, true>(a, go) : launch_join_as<R, false>(a, go);
}

template <int M, int P>
void launch_prompt(const PromptArgs& a, int waves, Launches& go) {
  const dim3 grid = wide_grid(((int64_t)a.items * a.heads + 7) / 8 * 8);          // a multiple of 8, up to 2^31 as wide too
  const size_t lds = 2 * PromptShape<M, P>::STAGE;
  if (waves == 8) go(prompt_kernel<M, P, 8>, grid, dim3(512), lds, a);
  else go(prompt_kernel<M, P, 4>, grid, dim3(256), lds, a);
}

}  // namespace

extern "C" {

fg_status fg_latent_attention_bytes(int32_t batch, int32_t heads, int32_t rank, int64_t* bytes) {
  if (!bytes || batch < 0 || batch > FG_ATTN_MAX_BATCH || heads < 1 || heads > FG_ATTN_MAX_HEADS || (rank != 256 && rank != 512)) return FG_EINVAL;
  const int64_t places = batch + latent_target(heads), tiles = (heads + 15) / 16;
  // absorbed queries; sums of the pieces; weighted means; pieces of every request
  *bytes = query_bytes(batch, heads, rank + 64) + (int64_t)batch * heads * 4 * rank + places * tiles * 16 * (4 * rank + 8) + 8 * (int64_t)batch;
  return FG_OK;
}

fg_status fg_latent_attention(const void* q, int64_t q_b, int64_t q_h, const void* w, const void* cache, int64_t page_stride,
                              int64_t row_stride, const fg_pages_t* pages, int32_t heads, int32_t rank, int32_t rope, int32_t nope,
                              float scale, void* workspace, int64_t workspace_bytes, void* out, int64_t out_b, int64_t out_h,
                              float* lse, int64_t lse_b, hipStream_t stream) {
  int64_t need = 0;
  if (!pages || !sizes_ok(heads, rank, rope, nope, scale) || fg_latent_attention_bytes(pages->batch, heads, rank, &need) != FG_OK) return FG_EINVAL;
  if (pages->n_pages < 1 || pages->page < 16 || pages->page % 16 || pages->width < 1 || pages->ldt < pages->width ||
      (int64_t)pages->width * pages->page > kMax)
    return FG_EINVAL;
  const int64_t batch = pages->batch, parts = head_parts(heads);
  // units of all requests are counted in 32 bits
  if (batch * ((int64_t)pages->width * pages->page / 32 + 2) > kMax) return FG_EINVAL;
  if (batch == 0) return FG_OK;
  if (!q || !w || !cache || !pages->table || !pages->lens || !out || !workspace || workspace_bytes < need) return FG_EINVAL;
  if (!aligned(q, 16) || !aligned(w, 16) || !aligned(cache, 16) || !aligned(out, 2) || !aligned(lse, 4) || !aligned(workspace, 16) ||
      !aligned(pages->table, 4) || !aligned(pages->lens, 4))
    return FG_EINVAL;
  if (!multiple(q_b, 8) || !multiple(q_h, 8) || !multiple(page_stride, 8) || !multiple(row_stride, 8) || 32 * row_stride > kMax || out_b < 0 || out_h < 0 ||
      (lse && lse_b < heads && batch > 1))
    return FG_EINVAL;
  if (!distinct({{batch, out_b}, {heads, out_h}, {nope, 1}})) return FG_EINVAL;
  const Rows ws = whole(workspace, need), o = rows3(out, 2, batch, out_b, heads, out_h, nope), qr = rows3(q, 2, batch, q_b, heads, q_h, nope + rope);
  const Rows cr = whole(cache, 2 * ((int64_t)(pages->n_pages - 1) * page_stride + (int64_t)(pages->page - 1) * row_stride + rank + rope));
  const Rows wr = whole(w, 4 * (int64_t)heads * nope * rank), le = whole(pages->lens, 4 * batch);
  const Rows t{pages->table, batch, 4 * (int64_t)pages->width, 4 * pages->ldt}, ls{lse, batch, 4 * (int64_t)heads, 4 * lse_b};
  if (overlaps(o, qr, wr, cr, t, le, ws, ls) || overlaps(ls, qr, wr, cr, t, le, ws) || overlaps(ws, qr, wr, cr, t, le)) return FG_EINVAL;
  const int64_t places = batch + latent_target(heads), tiles = (heads + 15) / 16;
  char* at = (char*)workspace;
  LatentArgs a{};
  char* const absorbed = at;
  at += query_bytes(batch, heads, rank + 64);
  a.part = (float*)at;
  at += places * tiles * 64 * rank;
  a.ml = (float*)at;
  at += places * tiles * 128;
  a.mean = (uint16_t*)at;
  at += batch * heads * 4 * rank;
  a.split = SplitArgs{pages->lens, pages->table, pages->ldt, pages->batch, pages->width, pages->n_pages, pages->page, 0, latent_target(heads),
                      (int32_t*)at};
  a.a = absorbed;
  a.rest = 2 * batch * heads * (rank + rope);
  a.cache = (const char*)cache;
  a.lse = lse;
  a.c_page = 2 * page_stride; a.c_tok = (int32_t)(2 * row_stride); a.lse_b = lse_b;
  a.heads = heads; a.tiles = (int32_t)tiles; a.parts = (int32_t)parts; a.c = scale * kLog2E;
  Launches go{stream};
  const unsigned b_tiles = (unsigned)((batch + 15) / 16);
  const AbsorbArgs absorb{(const char*)q, (const char*)w, absorbed, 2 * q_b, 2 * q_h, 4 * (int64_t)nope * rank, heads <= 16 ? a.rest : 0,
                          (int32_t)batch, heads, rank, rope};
  go(nope == 128 ? absorb_kernel<128> : absorb_kernel<64>, dim3((unsigned)rank / 128, (unsigned)heads, b_tiles), dim3(64), 0, absorb);
  const dim3 grid((unsigned)((a.split.target + 7) / 8 * 8 * parts));
  if (rank == 512) rope == 64 ? launch_latent<512, 64>(a, grid, go) : launch_latent<512, 32>(a, grid, go);
  else rope == 64 ? launch_latent<256, 64>(a, grid, go) : launch_latent<256, 32>(a, grid, go);
  rank == 512 ? launch_join<512>(a, go) : launch_join<256>(a, go);
  const ValuesArgs up{(const char*)a.mean, (const char*)w + 2 * (int64_t)nope * rank, (uint16_t*)out, 4 * (int64_t)nope * rank, out_b, out_h, (int32_t)batch, heads};
  const dim3 ug((unsigned)heads, (b_tiles + kValueTiles - 1) / kValueTiles);
  if (rank == 512) nope == 128 ? go(values_product_kernel<512, 128>, ug, dim3(512), values_lds(512), up) : go(values_product_kernel<512, 64>, ug, dim3(256), values_lds(512), up);
  else nope == 128 ? go(values_product_kernel<256, 128>, ug, dim3(512), values_lds(256), up) : go(values_product_kernel<256, 64>, ug, dim3(256), values_lds(256), up);
  return go.status();
}

fg_status fg_latent_prompt_bytes(int64_t k_rows, int32_t heads, int32_t nope, int64_t* bytes) {
  if (!bytes || k_rows < 0 || k_rows > kMax || heads < 1 || heads > FG_ATTN_MAX_HEADS || (nope != 64 && nope != 128)) return FG_EINVAL;
  *bytes = 4 * k_rows * heads * nope;
  return FG_OK;
}

fg_status fg_latent_prompt(const void* q, int64_t q_t, int64_t q_h, const int32_t* q_starts, int64_t q_rows, const void* latent,
                           int64_t ld, const int32_t* k_starts, int64_t k_rows, int32_t batch, const void* w, int32_t heads,
                           int32_t rank, int32_t rope, int32_t nope, float scale, void* workspace, int64_t workspace_bytes,
                           void* out, int64_t out_t, int64_t out_h, float* lse, int64_t lse_t, hipStream_t stream) {
  int64_t need = 0;
  if (!sizes_ok(heads, rank, rope, nope, scale) || fg_latent_prompt_bytes(k_rows, heads, nope, &need) != FG_OK || q_rows < 0 || q_rows > kMax - 1024 || batch < 0 ||
      batch > FG_ATTN_MAX_BATCH)
    return FG_EINVAL;
  if (batch == 0 || q_rows == 0) return FG_OK;
  if (!q || !q_starts || !k_starts || !w || !out || (k_rows && (!latent || !workspace)) || workspace_bytes < need) return FG_EINVAL;
  if (!aligned(q, 16) || !aligned(latent, 16) || !aligned(w, 16) || !aligned(q_starts, 4) || !aligned(k_starts, 4) || !aligned(out, 8) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return FG_EINVAL;
  if (!multiple(q_t, 8) || !multiple(q_h, 8) || !multiple(ld, 8) || (k_rows > 1 && ld < rank + rope) || 2 * ld >= 1 << 24 || !multiple(out_t, 4) || !multiple(out_h, 4) ||
      (lse && lse_t < heads && q_rows > 1))
    return FG_EINVAL;
  if (!distinct({{q_rows, out_t}, {heads, out_h}, {nope, 1}})) return FG_EINVAL;
  const Rows ws = whole(k_rows ? workspace : nullptr, need), o = rows3(out, 2, q_rows, out_t, heads, out_h, nope), qr = rows3(q, 2, q_rows, q_t, heads, q_h, nope + rope);
  const Rows lat = {k_rows ? latent : nullptr, k_rows, 2 * (int64_t)(rank + rope), 2 * ld}, wr = whole(w, 4 * (int64_t)heads * nope * rank);
  const Rows qs = whole(q_starts, 4 * ((int64_t)batch + 1)), ks = whole(k_starts, 4 * ((int64_t)batch + 1)), ls{lse, q_rows, 4 * (int64_t)heads, 4 * lse_t};
  if (overlaps(o, qr, lat, wr, qs, ks, ws, ls) || overlaps(ls, qr, lat, wr, qs, ks, ws) || overlaps(ws, qr, lat, wr, qs, ks)) return FG_EINVAL;
  // tiles of 256 queries where they fill the GPU twice, else of 128
  const int waves = (q_rows + 255) / 256 * heads >= 2 * kCUs ? 8 : 4;
  const int64_t items = (q_rows + 32 * waves - 1) / (32 * waves) + batch, n = (int64_t)heads * 2 * nope;
  if (items * heads > kMax - 8 || (k_rows + kExpandTile - 1) / kExpandTile > 65535 || n > kMax) return FG_EINVAL;
  Launches go{stream};
  if (k_rows) {
    const ExpandArgs e{(const char*)latent, (const char*)w, (uint16_t*)workspace, 2 * ld, k_rows, (int32_t)n, rank};
    go(expand_kernel, dim3((unsigned)(n / kExpandTile), (unsigned)((k_rows + kExpandTile - 1) / kExpandTile)), dim3(256), kExpandStages * kExpandStage, e);
  }
  PromptArgs a{};
  a.q = (const char*)q; a.kv = (const char*)workspace; a.lat = (const char*)latent; a.out = (uint16_t*)out; a.lse = lse;
  a.q_starts = q_starts; a.k_starts = k_starts;
  a.q_t = 2 * q_t; a.q_h = 2 * q_h; a.ld = 2 * ld; a.out_t = out_t; a.out_h = out_h; a.lse_t = lse_t;
  a.q_rows = q_rows; a.k_rows = k_rows; a.batch = batch; a.heads = heads; a.r = rank; a.items = (int32_t)items; a.c = scale * kLog2E;
  if (nope == 128) rope == 64 ? launch_prompt<128, 64>(a, waves, go) : launch_prompt<128, 32>(a, waves, go);
  else rope == 64 ? launch_prompt<64, 64>(a, waves, go) : launch_prompt<64, 32>(a, waves, go);
  return go.status();
}

}  // extern "C"
