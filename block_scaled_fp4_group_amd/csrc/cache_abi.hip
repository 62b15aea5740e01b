// C entry points of the calls around the cache -- held in 4 bits, its pages, its rows
// read back -- and of the residual stream's norms: argument checks, then launches.
#include "attn_check.h"

namespace moe {

moe_status launch_qk_norm_rope_fp4(const moe_heads&, const moe_heads&, const moe_heads&, int64_t, const moe_rope_params&,
                                   const int32_t*, const float*, const float*, const float*, const moe_heads&,
                                   const moe_heads*, const moe_kv_cache_fp4&, const int32_t*, hipStream_t);
moe_status launch_kv_gather(const moe_kv_cache&, int, int, int, const int32_t*, int64_t, int, const int32_t*, int64_t,
                            const int32_t*, int, int64_t, const moe_heads&, const moe_heads&, hipStream_t);
moe_status launch_kv_gather_fp4(const moe_kv_cache_fp4&, int, int, int, const int32_t*, int64_t, int, const int32_t*, int64_t,
                                const int32_t*, int, int64_t, const moe_heads&, const moe_heads&, hipStream_t);
int64_t kv_gather_grid(int64_t, int);
int64_t qk_norm_rope_fp4_threads(int64_t, const moe_rope_params&);
size_t attn_decode_fp4_ws_bytes(int64_t, const moe_attn_params&, int64_t, int64_t);
int64_t attn_decode_fp4_threads(int64_t, const moe_attn_params&, int64_t, int64_t);
moe_status launch_attn_decode_fp4(const moe_heads&, const moe_kv_cache_fp4&, const int32_t*, int64_t, const int32_t*, int64_t,
                                  int64_t, const int32_t*, int64_t, const moe_attn_params&, const moe_heads&, float*, void*,
                                  hipStream_t);
int64_t kv_pages_most();
size_t kv_compact_ws_bytes(int64_t);
moe_status launch_kv_fork(int32_t*, int64_t, int, int, int32_t*, const int32_t*, const int32_t*, int, const int32_t*, int64_t,
                          int, const moe_page_buffers&, int64_t, int32_t*, hipStream_t);
size_t kv_free_ws_bytes(int64_t, int64_t, int64_t);
moe_status launch_kv_free_pages(const int32_t*, int64_t, int, int, const int32_t*, int, int64_t, int32_t*, int32_t*, void*,
                                hipStream_t);
moe_status launch_kv_compact(const int32_t*, int64_t, int, int, const int32_t*, int, const moe_page_buffers&, int64_t, int32_t*,
                             int64_t, int32_t*, void*, hipStream_t);
int block_norm_max_hidden();
moe_status launch_block_norm(const moe_rows&, int64_t, int, const moe_rows*, const float*, const moe_rows*, const float*, float,
                             const float*, float, const moe_rows*, const moe_rows*, hipStream_t);

static moe_status check_cache_fp4(const char* fn, const moe_kv_cache_fp4* c) {
  MOE_CHECK(c && c->k && c->v && c->k_scale && c->v_scale, "%s: cache is NULL", fn);
  MOE_CHECK(aligned16(c->k) && aligned16(c->v) && aligned16(c->k_scale) && aligned16(c->v_scale),
            "%s: cache must be 16-byte aligned", fn);
  MOE_CHECK(is_pow2_int(c->page_size) && c->page_size >= 16 && c->page_size <= 1024,
            "%s: page_size %d is no power of two from 16 to 1024", fn, c->page_size);
  MOE_CHECK(c->num_pages >= 1 && c->num_pages <= (int64_t)0x7fffffff / c->page_size,
            "%s: num_pages outside [1, 2^31 / page_size)", fn);
  for (const float g : {c->k_global, c->v_global}) {
    int e;
    MOE_CHECK(std::isfinite(g) && g > 0.0f && std::frexp(g, &e) == 0.5f && e >= -31 && e <= 33,
              "%s: the global scales must be powers of two from 2^-32 to 2^32", fn);
  }
  return MOE_OK;
}

static moe_status check_table(const char* fn, const int32_t* table, int64_t stride, int32_t rows, int32_t max_blocks,
                              const int32_t* lens, int32_t page_size, int64_t num_pages) {
  MOE_CHECK(rows >= 0 && max_blocks >= 0, "%s: negative size", fn);
  MOE_CHECK(is_pow2_int(page_size) && page_size <= 1024, "%s: page_size %d is no power of two up to 1024", fn, page_size);
  MOE_CHECK((int64_t)max_blocks * page_size <= 0x7fffffff && stride >= max_blocks, "%s: bad max_blocks / table_stride", fn);
  MOE_CHECK(rows == 0 || max_blocks == 0 || (table && lens), "%s: block_table or lens is NULL", fn);
  MOE_CHECK(num_pages >= 1 && num_pages <= (int64_t)0x7fffffff / page_size, "%s: num_pages outside [1, 2^31 / page_size)", fn);
  return MOE_OK;
}

static moe_status check_pool(const char* fn, int64_t num_pages) {
  if (num_pages <= kv_pages_most()) return MOE_OK;
  set_error("%s: %lld pages, at most %lld", fn, (long long)num_pages, (long long)kv_pages_most());
  return MOE_ERR_UNSUPPORTED;
}

static moe_status check_workspace(const char* fn, const void* workspace, size_t bytes, size_t need) {
  if (need == 0 || (workspace != nullptr && bytes >= need && aligned16(workspace))) return MOE_OK;
  set_error("%s: workspace %zu bytes < %zu (or NULL / unaligned)", fn, bytes, need);
  return MOE_ERR_WORKSPACE;
}

static moe_status check_buffers(const char* fn, const moe_page_buffers* b) {
  MOE_CHECK(b && b->count >= 0 && b->count <= MOE_PAGE_BUFFERS, "%s: up to %d page buffers", fn, MOE_PAGE_BUFFERS);
  for (int i = 0; i < b->count; ++i)
    MOE_CHECK(b->data[i] && aligned16(b->data[i]) && b->page_bytes[i] > 0 && b->page_bytes[i] % 16 == 0 &&
                  b->page_bytes[i] <= ((int64_t)1 << 40),
              "%s: page buffer %d is NULL, or it or its pages are not multiples of 16 bytes", fn, i);
  return MOE_OK;
}

// rows of `hidden` bf16; written ones must not overlap
static moe_status check_rows(const char* fn, const char* name, const moe_rows* x, int64_t T, int32_t hidden, bool written) {
  MOE_CHECK(x->data && aligned16(x->data) && x->stride % 8 == 0 && x->stride >= 0,
            "%s: %s needs 16-byte alignment and a stride that is a multiple of 8 elements", fn, name);
  MOE_CHECK(!written || T <= 1 || x->stride >= hidden, "%s: rows of %s overlap", fn, name);
  return MOE_OK;
}

static moe_status check_gather(const char* fn, int32_t kv_heads, int32_t k_dim, int32_t v_dim, const int32_t* block_table,
                               int64_t table_stride, int32_t max_blocks, const int32_t* prefix_table, int32_t prefix_blocks,
                               int64_t prefix_len, int32_t page_size, const int32_t* cu_k, int32_t num_seqs, int64_t total_k,
                               const moe_heads* k_out, const moe_heads* v_out) {
  MOE_CHECK(kv_heads >= 1 && kv_heads <= 65536 && k_dim >= 16 && k_dim <= 1024 && k_dim % 16 == 0 && v_dim >= 16 &&
                v_dim <= 1024 && v_dim % 16 == 0,
            "%s: head sizes must be multiples of 16 up to 1024", fn);
  MOE_CHECK(max_blocks >= 0 && prefix_blocks >= 0 && prefix_len >= 0, "%s: negative size", fn);
  MOE_CHECK(cu_k, "%s: cu_k is NULL", fn);
  MOE_CHECK(total_k <= 0x7fffffff, "%s: over 2^31 - 1 rows", fn);
  MOE_CHECK(launch_fits(kv_gather_grid(total_k, kv_heads), 256), "%s: too many rows", fn);
  MOE_CHECK(table_stride >= max_blocks && (max_blocks == 0 || block_table), "%s: block_table NULL or its stride too small", fn);
  MOE_CHECK(prefix_len <= (int64_t)prefix_blocks * page_size, "%s: prefix_len %lld needs more than %d pages", fn,
            (long long)prefix_len, prefix_blocks);
  MOE_CHECK(prefix_len == 0 || prefix_table, "%s: prefix_table is NULL", fn);
  MOE_PASS(check_heads(fn, "k_out", k_out, kv_heads, k_dim, total_k));
  return check_heads(fn, "v_out", v_out, kv_heads, v_dim, total_k);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_qk_norm_rope_fp4(const moe_heads* q, const moe_heads* k, const moe_heads* v, int64_t T,
                                const moe_rope_params* p, const int32_t* positions, const float* cos_sin,
                                const float* q_weight, const float* k_weight, const moe_heads* q_out,
                                const moe_heads* k_out, const moe_kv_cache_fp4* cache, const int32_t* slots,
                                hipStream_t stream) {
  const char* fn = "moe_qk_norm_rope_fp4";
  set_error("");
  MOE_PASS(check_rope(fn, T, p));
  // a block of 16 values lies in two lanes, which hold both halves of every pair
  if (p->rot_dim % 32 != 0) {
    set_error("%s: rot_dim %d is no multiple of 32", fn, p->rot_dim);
    return MOE_ERR_UNSUPPORTED;
  }
  MOE_CHECK(p->v_dim >= 16 && p->v_dim % 16 == 0, "%s: v_dim %d is no positive multiple of 16", fn, p->v_dim);
  if (T == 0) return MOE_OK;
  MOE_PASS(check_rope_data(fn, T, p, q, k, positions, cos_sin, q_weight, k_weight, q_out, k_out));
  MOE_PASS(check_cache_fp4(fn, cache));
  MOE_CHECK(slots, "%s: slots is NULL", fn);
  MOE_PASS(check_heads(fn, "v", v, p->kv_heads, p->v_dim, 0));
  MOE_CHECK(launch_fits(qk_norm_rope_fp4_threads(T, *p), 1), "%s: too many heads", fn);
  return launch_qk_norm_rope_fp4(*q, *k, *v, T, *p, positions, cos_sin, q_weight, k_weight, *q_out, k_out, *cache, slots,
                                 stream);
}

size_t moe_attn_decode_fp4_workspace_bytes(int32_t num_requests, int64_t prefix_len, int64_t max_len,
                                           const moe_attn_params* p) {
  if (!sizes_of_heads(p) || num_requests <= 0 || prefix_len < 0 || max_len < 0 ||
      !decode_sizes_fit(num_requests, prefix_len, max_len, *p))
    return 0;
  return attn_decode_fp4_ws_bytes(num_requests, *p, prefix_len, max_len);
}

moe_status moe_attn_decode_fp4(const moe_heads* q, const moe_kv_cache_fp4* cache, const int32_t* block_table,
                               int64_t table_stride, int32_t max_blocks, const int32_t* lens, int32_t num_requests,
                               int64_t max_len, const int32_t* prefix_table, int32_t prefix_blocks, int64_t prefix_len,
                               const moe_attn_params* p, const moe_heads* out, float* lse, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "moe_attn_decode_fp4";
  set_error("");
  MOE_PASS(check_attn(fn, p));
  MOE_CHECK(num_requests >= 0 && max_len >= 0 && prefix_len >= 0 && max_blocks >= 0 && prefix_blocks >= 0,
            "%s: negative size", fn);
  if (num_requests == 0) return MOE_OK;
  MOE_PASS(check_cache_fp4(fn, cache));
  MOE_PASS(check_heads(fn, "q", q, p->q_heads, p->k_dim, 0));
  MOE_PASS(check_heads(fn, "out", out, p->q_heads, p->v_dim, num_requests));
  MOE_CHECK(lens, "%s: lens is NULL", fn);
  MOE_CHECK(max_len <= (int64_t)max_blocks * cache->page_size, "%s: max_len %lld needs more than max_blocks %d pages", fn,
            (long long)max_len, max_blocks);
  MOE_CHECK(max_len == 0 || (block_table && table_stride >= max_blocks), "%s: block_table NULL or its stride too small",
            fn);
  MOE_CHECK(prefix_len <= (int64_t)prefix_blocks * cache->page_size, "%s: prefix_len %lld needs more than %d pages", fn,
            (long long)prefix_len, prefix_blocks);
  MOE_CHECK(prefix_len == 0 || prefix_table, "%s: prefix_table is NULL", fn);
  MOE_CHECK(decode_sizes_fit(num_requests, prefix_len, max_len, *p), "%s: too many keys or rows", fn);
  MOE_CHECK(aligned4(lse), "%s: lse not 4-byte aligned", fn);
  MOE_CHECK(launch_fits(attn_decode_fp4_threads(num_requests, *p, prefix_len, max_len), 1), "%s: too many rows", fn);
  MOE_PASS(check_workspace(fn, workspace, workspace_bytes, attn_decode_fp4_ws_bytes(num_requests, *p, prefix_len, max_len)));
  return launch_attn_decode_fp4(*q, *cache, block_table, table_stride, lens, num_requests, max_len, prefix_table, prefix_len,
                                *p, *out, lse, workspace, stream);
}

moe_status moe_kv_gather(const moe_kv_cache* cache, int32_t kv_heads, int32_t k_dim, int32_t v_dim,
                         const int32_t* block_table, int64_t table_stride, int32_t max_blocks, const int32_t* prefix_table,
                         int32_t prefix_blocks, int64_t prefix_len, const int32_t* cu_k, int32_t num_seqs, int64_t total_k,
                         const moe_heads* k_out, const moe_heads* v_out, hipStream_t stream) {
  const char* fn = "moe_kv_gather";
  set_error("");
  MOE_CHECK(num_seqs >= 0 && total_k >= 0, "%s: negative size", fn);
  if (num_seqs == 0 || total_k == 0) return MOE_OK;
  MOE_PASS(check_cache(fn, cache));
  MOE_PASS(check_gather(fn, kv_heads, k_dim, v_dim, block_table, table_stride, max_blocks, prefix_table, prefix_blocks,
                        prefix_len, cache->page_size, cu_k, num_seqs, total_k, k_out, v_out));
  return launch_kv_gather(*cache, kv_heads, k_dim, v_dim, block_table, table_stride, max_blocks, prefix_table, prefix_len,
                          cu_k, num_seqs, total_k, *k_out, *v_out, stream);
}

moe_status moe_kv_gather_fp4(const moe_kv_cache_fp4* cache, int32_t kv_heads, int32_t k_dim, int32_t v_dim,
                             const int32_t* block_table, int64_t table_stride, int32_t max_blocks,
                             const int32_t* prefix_table, int32_t prefix_blocks, int64_t prefix_len, const int32_t* cu_k,
                             int32_t num_seqs, int64_t total_k, const moe_heads* k_out, const moe_heads* v_out,
                             hipStream_t stream) {
  const char* fn = "moe_kv_gather_fp4";
  set_error("");
  MOE_CHECK(num_seqs >= 0 && total_k >= 0, "%s: negative size", fn);
  if (num_seqs == 0 || total_k == 0) return MOE_OK;
  MOE_PASS(check_cache_fp4(fn, cache));
  MOE_PASS(check_gather(fn, kv_heads, k_dim, v_dim, block_table, table_stride, max_blocks, prefix_table, prefix_blocks,
                        prefix_len, cache->page_size, cu_k, num_seqs, total_k, k_out, v_out));
  return launch_kv_gather_fp4(*cache, kv_heads, k_dim, v_dim, block_table, table_stride, max_blocks, prefix_table, prefix_len,
                              cu_k, num_seqs, total_k, *k_out, *v_out, stream);
}

moe_status moe_kv_fork(int32_t* block_table, int64_t table_stride, int32_t num_rows, int32_t max_blocks, int32_t* lens,
                       const int32_t* parents, const int32_t* children, int32_t num_forks, const int32_t* free_pages,
                       int64_t num_free, int32_t page_size, const moe_page_buffers* buffers, int64_t num_pages,
                       int32_t* counts, hipStream_t stream) {
  const char* fn = "moe_kv_fork";
  set_error("");
  MOE_PASS(check_table(fn, block_table, table_stride, num_rows, max_blocks, lens, page_size, num_pages));
  MOE_PASS(check_buffers(fn, buffers));
  MOE_CHECK(num_forks >= 0 && num_free >= 0, "%s: negative size", fn);
  if (num_forks > (1 << 16)) {
    set_error("%s: %d forks, at most %d", fn, num_forks, 1 << 16);
    return MOE_ERR_UNSUPPORTED;
  }
  MOE_CHECK(num_forks == 0 || (parents && children), "%s: parents or children is NULL", fn);
  MOE_CHECK(num_free == 0 || free_pages, "%s: free_pages is NULL", fn);
  MOE_CHECK(counts, "%s: counts is NULL", fn);
  return launch_kv_fork(block_table, table_stride, max_blocks == 0 ? 0 : num_rows, max_blocks, lens, parents, children, num_forks, free_pages, num_free,
                        __builtin_ctz((unsigned)page_size), *buffers, num_pages, counts, stream);
}

size_t moe_kv_free_pages_workspace_bytes(int32_t num_rows, int32_t max_blocks, int64_t num_pages) {
  return num_rows < 0 || max_blocks < 0 || num_pages < 1 || num_pages > kv_pages_most() ? 0
                                                                                       : kv_free_ws_bytes(num_rows, max_blocks, num_pages);
}

moe_status moe_kv_free_pages(const int32_t* block_table, int64_t table_stride, int32_t num_rows, int32_t max_blocks,
                             const int32_t* lens, int32_t page_size, int64_t num_pages, int32_t* free_pages, int32_t* counts,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "moe_kv_free_pages";
  set_error("");
  MOE_PASS(check_table(fn, block_table, table_stride, num_rows, max_blocks, lens, page_size, num_pages));
  MOE_PASS(check_pool(fn, num_pages));
  MOE_CHECK(free_pages && counts, "%s: free_pages or counts is NULL", fn);
  MOE_PASS(check_workspace(fn, workspace, workspace_bytes, kv_free_ws_bytes(num_rows, max_blocks, num_pages)));
  return launch_kv_free_pages(block_table, table_stride, max_blocks == 0 ? 0 : num_rows, max_blocks, lens,
                              __builtin_ctz((unsigned)page_size), num_pages, free_pages, counts, workspace, stream);
}

size_t moe_kv_compact_workspace_bytes(int64_t num_pages) {
  return num_pages < 1 || num_pages > kv_pages_most() ? 0 : kv_compact_ws_bytes(num_pages);
}

moe_status moe_kv_compact(const int32_t* block_table, int64_t table_stride, int32_t num_rows, int32_t max_blocks,
                          const int32_t* lens, int32_t page_size, const moe_page_buffers* buffers, int64_t num_pages,
                          int32_t* out_table, int64_t out_stride, int32_t* counts, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
  const char* fn = "moe_kv_compact";
  set_error("");
  MOE_PASS(check_table(fn, block_table, table_stride, num_rows, max_blocks, lens, page_size, num_pages));
  MOE_PASS(check_pool(fn, num_pages));
  MOE_PASS(check_buffers(fn, buffers));
  MOE_CHECK(out_stride >= max_blocks && (num_rows == 0 || max_blocks == 0 || out_table), "%s: out_table NULL or its stride too small", fn);
  MOE_CHECK(counts, "%s: counts is NULL", fn);
  if (num_rows > 0 && max_blocks > 0) {
    // the table itself, row by row, or another place
    const int64_t n = num_rows - 1;
    MOE_CHECK((out_table == block_table && (num_rows == 1 || out_stride == table_stride)) ||
                  out_table + n * out_stride + max_blocks <= block_table || block_table + n * table_stride + max_blocks <= out_table,
              "%s: out_table overlaps block_table", fn);
  }
  MOE_PASS(check_workspace(fn, workspace, workspace_bytes, kv_compact_ws_bytes(num_pages)));
  return launch_kv_compact(block_table, table_stride, max_blocks == 0 ? 0 : num_rows, max_blocks, lens,
                           __builtin_ctz((unsigned)page_size), *buffers, num_pages, out_table, out_stride, counts, workspace,
                           stream);
}

moe_status moe_block_norm(const moe_rows* x, int64_t T, int32_t hidden, const moe_rows* residual, const float* post_weight,
                          const moe_rows* gate, const float* channel_gate, float scale, const float* weight, float eps,
                          const moe_rows* h, const moe_rows* y, hipStream_t stream) {
  const char* fn = "moe_block_norm";
  set_error("");
  MOE_CHECK(T >= 0 && T <= 0x7fffffff, "%s: bad number of rows", fn);
  MOE_CHECK(hidden >= 8 && hidden % 8 == 0, "%s: hidden %d is no positive multiple of 8", fn, hidden);
  if (hidden > block_norm_max_hidden()) {
    set_error("%s: hidden %d, at most %d", fn, hidden, block_norm_max_hidden());
    return MOE_ERR_UNSUPPORTED;
  }
  MOE_CHECK(std::isfinite(scale), "%s: scale must be finite", fn);
  MOE_CHECK(eps >= 0.0f && std::isfinite(eps), "%s: eps must be finite and not negative", fn);
  MOE_CHECK(h || y, "%s: neither h nor y is asked for", fn);
  MOE_CHECK(!y || weight, "%s: y needs weight", fn);
  MOE_CHECK(!gate || !channel_gate, "%s: a gate of each value or of each channel, not both", fn);
  MOE_CHECK((!weight || aligned16(weight)) && (!post_weight || aligned16(post_weight)) &&
                (!channel_gate || aligned16(channel_gate)),
            "%s: weights must be 16-byte aligned", fn);
  if (T == 0) return MOE_OK;
  MOE_CHECK(x, "%s: x is NULL", fn);
  MOE_PASS(check_rows(fn, "x", x, T, hidden, false));
  if (residual) MOE_PASS(check_rows(fn, "residual", residual, T, hidden, false));
  if (gate) MOE_PASS(check_rows(fn, "gate", gate, T, hidden, false));
  if (h) MOE_PASS(check_rows(fn, "h", h, T, hidden, true));
  if (y) MOE_PASS(check_rows(fn, "y", y, T, hidden, true));
  return launch_block_norm(*x, T, hidden, residual, post_weight, gate, channel_gate, scale, weight, eps, h, y, stream);
}

}  // extern "C"
