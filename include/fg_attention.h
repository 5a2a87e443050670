/*
 * fg_attention.h -- the attention half of a decoder layer for serving, over a paged
 * cache: pages and slots of a step, rows written to their slots, attention of one
 * new token, and attention whose keys and values come from one latent vector a
 * token (absorbed form for one new token, expanded form for prompts). They stand
 * beside the decoding operators of fg.h and follow their conventions: no context,
 * a few kernels on `stream` (of the current device), nothing allocated or kept, all
 * may be captured into a graph; pointers are device pointers owned by the caller;
 * errors FG_EINVAL (shapes, types, NULLs, alignment, outputs on memory that is
 * still read) and FG_EHIP (a launch failed). Rows, requests of 0: FG_OK, nothing is
 * launched (but by fg_page_step, which has outputs without them too). Results do not depend on timing.
 *
 * The cache: n_pages pages of `page` rows (tokens), page a multiple of 16. A request's
 * token t lies in row t % page of page table[request][t / page]. Strides are in
 * elements; pages, tokens and heads may lie in any order, the columns of a row
 * are consecutive. A slot is page number * page + row.
 *
 * In all attention here a request's numbers of tokens and pages are read on the GPU. Entries of
 * `table` behind a request's last token are not read; a page number outside
 * 0..n_pages-1 leaves its tokens out, as if they were not there. A row that sees no token gives zeros and
 * an lse of -infinity, and so does one whose scores are all -infinity. What lies in the cache behind a
 * request's last token, before its window or on other pages, NaN and infinities
 * included, does not reach its results; a NaN or an infinity among the tokens
 * that it sees gives what the formula gives, or NaN. lse is log(sum exp(scale s)) over the tokens seen,
 * by which results of parts of a cache can be joined.
 * Scores, maxima and sums are fp32; a token's weight is rounded to bf16 (2^-8 relative at most) before it
 * multiplies the value, and the result is rounded once. Weights are up to 2^8 and are divided by their sum at the
 * end, so a value times the number of tokens has to stay below 2^120.
 */
#ifndef FG_ATTENTION_H
#define FG_ATTENTION_H

#include "fg.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FG_ATTN_MAX_BATCH 65535
#define FG_ATTN_MAX_HEADS 65535
#define FG_APPEND_MAX_DIM 1024          /* 8-bit caches */

/* One scheduling step of `batch` requests, in order: add[b] > 0 asks for that many
 * new tokens, 0 leaves the request alone, < 0 ends it (its pages go back to the
 * ring and its length becomes 0). Free pages wait in `ring`: number `i` from the start
 * of time is ring[i mod n_pages], those with ends[0] <= i < ends[1] are free; both numbers only ever grow.
 *   held = ceil(len / page), wants = ceil((len + add) / page)
 * A request is served when wants <= width, and its pages up to and including
 * its own, summed over the requests that fit their table, are free (or it needs none),
 * and the tokens of the requests that have their pages, up to and including its own, are
 * no more than `tokens`. One that is not keeps its length and gets no slots; nothing else tells.
 * Served requests take pages from the ring in order, into table[b][held..wants-1]. Pages that
 * come back in this step can be taken in the next one.
 *   lens_out[b] = len + add (0 when it has ended);  ends_out: the ring afterwards
 *   starts[b]:  tokens of the served requests before b; starts[batch] their sum
 *   slots, positions: for token j of request b at starts[b] + j: its slot (-1 on a page number < 0) and
 *               len + j; -1 and 0 from starts[batch] to tokens - 1
 *   lens, add:  int32 [batch] (a length < 0 counts as 0);  table: int32 [batch][ldt], width columns, written
 *   ring:       int32 [n_pages], written;  ends: int64 [2]
 *   lens_out:   int32 [batch], may be lens;  ends_out: int64 [2], may be ends
 *   starts:     int32 [batch + 1];  slots: int64 [tokens];  positions: int32 [tokens]
 *   page >= 1 (here); width * page < 2^31. No other two may share memory. With batch 0 only starts, ends and
 *   the outputs of `tokens` are needed: starts[0] = 0, ends_out = ends. */
fg_status fg_page_step(const int32_t* lens, const int32_t* add, int32_t batch, int32_t* table, int64_t ldt, int32_t width,
                       int32_t* ring, const int64_t* ends, int32_t n_pages, int32_t page, int32_t* lens_out, int64_t* ends_out,
                       int32_t* starts, int64_t* slots, int32_t* positions, int32_t tokens, hipStream_t stream);

/* Write new rows to their slots: cache[slot / page][slot % page][h] = x[i][h] for each
 * of keys and values (values may be NULL: one kind of rows, as latents are).
 *   x:      bf16 [rows][heads][dim] with strides
 *   cache:  FG_BF16: the same bits; FG_E4M3: with a = max |x[i][h]| the scale a / 448 and
 *           codes rne(448 x / a) of the exact quotient, 0 where a = 0 (a NaN or an infinity makes the scale NaN or infinite)
 *   scale:  fp32 [n_pages][heads][page], FG_E4M3 only
 *   slots:  int64 [rows], distinct; a row whose slot is outside 0..n_pages * page - 1 is skipped
 *   dim a multiple of 8; rows of x and of a bf16 cache start on 16-byte, of an e4m3 cache on 8-byte
 *   boundaries (strides multiples of 8). Inputs and caches share no memory. Caches of keys and values may lie
 *   within each other if their strides are equal, or page beside page. */
typedef struct {
  const void* x;                        /* new rows */
  int64_t x_row, x_head;
  void* cache;
  int64_t page_stride, row_stride, head_stride;
  float* scale;
} fg_append_t;
fg_status fg_kv_append(const fg_append_t* keys, const fg_append_t* values, int32_t cache_type, const int64_t* slots, int64_t rows,
                       int32_t heads, int32_t dim, int32_t n_pages, int32_t page, hipStream_t stream);

/* A paged cache and the requests in it, as the attention reads them. */
typedef struct {
  const int32_t* table;                 /* int32 [batch][ldt], width columns */
  int64_t ldt;
  int32_t width;
  const int32_t* lens;                  /* int32 [batch]: tokens in the cache, the new one among them; at most width * page count */
  int32_t batch;
  int32_t n_pages, page;
} fg_pages_t;

/* Attention of one new token a request; its own key and value are in the cache.
 *   out[b][h] = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale q[b][h] . k_t),  t over the last `window`
 *   tokens of the request (window 0: all), k and v those of head h / group
 * Split over the cache's length into pieces that fill the GPU, joined by a second kernel.
 *   q:      bf16 [batch][kv * group][dim], heads of one key together; rows on 16-byte boundaries
 *   k, v:   bf16 or e4m3 [n_pages][page][kv][dim], rows on 16-byte boundaries, strides multiples of 8 (16 for e4m3);
 *           16 rows of a page are less than 2^31 bytes apart
 *   scales: fp32 [n_pages][kv][page] for e4m3 (the code times its scale is the value), 16-byte aligned
 *   dim 64, 128 or 256; scale > 0; width * page < 2^31, batch * width * page < 2^38 - 2^9 * batch
 *   out:    bf16 [batch][kv * group][dim], rows consecutive (out_b, out_h >= dim);  lse: fp32 [batch][kv * group] or NULL
 *   workspace: fg_paged_attention_bytes, 16-byte aligned, contents free; calls that may overlap need one each */
typedef struct {
  const void* data;
  int64_t page_stride, row_stride, head_stride;
  const float* scale;
} fg_cache_t;
fg_status fg_paged_attention_bytes(int32_t batch, int32_t kv, int32_t group, int32_t dim, int64_t* bytes);
fg_status fg_paged_attention(const void* q, int64_t q_b, int64_t q_h, const fg_cache_t* k, const fg_cache_t* v, int32_t cache_type,
                             const fg_pages_t* pages, int32_t kv, int32_t group, int32_t dim, int32_t window, float scale,
                             void* workspace, int64_t workspace_bytes, void* out, int64_t out_b, int64_t out_h, float* lse,
                             int64_t lse_b, hipStream_t stream);

/* Latent attention. A token has one row [latent c of `rank` | rotary key r of `rope`] for all
 * heads; head h has the weights W_k = w[h][0..nope-1], W_v = w[h][nope..2 nope-1], rows of `rank`:
 *   keys [W_k c | r], values W_v c;  queries [q_nope | q_rope], q_rope already turned
 * rank 256 or 512, rope 32 or 64, nope 64 or 128 (columns of a value as well); w bf16
 * [heads][2 nope][rank], contiguous, 16-byte aligned; scale > 0.
 *
 * fg_latent_attention: the absorbed form of one new token a request, over a paged cache of
 * rows: the score of a token is scale ((W_k^T q_nope) . c + q_rope . r), the result W_v applied to the
 * weighted mean of c. W_k^T q_nope is rounded to bf16 before its product,
 * or held as two bf16 numbers, within 2^-16, where there are up to 16 heads; so is the mean, and so are the weights of up to 32 heads.
 *   q:      bf16 [batch][heads][nope + rope], rows on 16-byte boundaries
 *   cache:  bf16 [n_pages][page][rank + rope] rows on 16-byte boundaries (strides multiples of 8, 16 rows less than 2^31 bytes apart);
 *           width * page < 2^31, batch * width * page < 2^36 - 2^7 * batch
 *   out:    bf16 [batch][heads][nope];  lse: fp32 [batch][heads] or NULL
 *   workspace: fg_latent_attention_bytes, 16-byte aligned */
fg_status fg_latent_attention_bytes(int32_t batch, int32_t heads, int32_t rank, int64_t* bytes);
fg_status fg_latent_attention(const void* q, int64_t q_b, int64_t q_h, const void* w, const void* cache, int64_t page_stride,
                              int64_t row_stride, const fg_pages_t* pages, int32_t heads, int32_t rank, int32_t rope, int32_t nope,
                              float scale, void* workspace, int64_t workspace_bytes, void* out, int64_t out_b, int64_t out_h,
                              float* lse, int64_t lse_b, hipStream_t stream);

/* fg_latent_prompt: the expanded form for `batch` requests one after the other. Request b has the
 * queries q_starts[b]..q_starts[b + 1]-1, which are the last tokens of its keys
 * k_starts[b]..k_starts[b + 1]-1; query i of nq sees keys 0..nk - nq + i of nk. Keys and values are
 * formed once, rounded to bf16, in the workspace. A NaN or an infinity in a row that a query does not see does not reach it.
 *   q:      bf16 [q_rows][heads][nope + rope], rows on 16-byte boundaries
 *   latent: bf16 [k_rows][ld], rank + rope columns, rows on 16-byte boundaries, less than 2^24 bytes apart
 *   k_rows <= 65535 * 128, q_rows < 2^31 - 1024, (q_rows / 128 + batch + 1) * heads < 2^31 - 8, heads * 2 nope < 2^31
 *   starts: int32 [batch + 1], not falling; one outside 0..q_rows, 0..k_rows counts as the nearest of these
 *   out:    bf16 [q_rows][heads][nope], strides multiples of 4, 8-byte aligned; rows of no request are left as they were
 *   lse:    fp32 [q_rows][heads] or NULL
 *   workspace: fg_latent_prompt_bytes, 16-byte aligned */
fg_status fg_latent_prompt_bytes(int64_t k_rows, int32_t heads, int32_t nope, int64_t* bytes);
fg_status fg_latent_prompt(const void* q, int64_t q_t, int64_t q_h, const int32_t* q_starts, int64_t q_rows, const void* latent,
                           int64_t ld, const int32_t* k_starts, int64_t k_rows, int32_t batch, const void* w, int32_t heads,
                           int32_t rank, int32_t rope, int32_t nope, float scale, void* workspace, int64_t workspace_bytes,
                           void* out, int64_t out_t, int64_t out_h, float* lse, int64_t lse_t, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FG_ATTENTION_H */
