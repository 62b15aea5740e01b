// C entry points of the attention operators: argument checks, then launches.
#include "attn_check.h"

namespace moe {

int kv_slots_max_requests();
moe_status launch_kv_slots(const int32_t*, const int32_t*, int, const int32_t*, int64_t, int, int32_t*, int64_t, int, int,
                           int64_t, int32_t*, int32_t*, int32_t*, int32_t*, hipStream_t);
moe_status launch_qk_norm_rope(const moe_heads&, const moe_heads&, const moe_heads*, int64_t, const moe_rope_params&,
                               const int32_t*, const float*, const float*, const float*, const moe_heads&,
                               const moe_heads*, const moe_kv_cache*, const int32_t*, hipStream_t);
moe_status launch_attn_prompt(const moe_heads&, const moe_heads&, const moe_heads&, const int32_t*, const int32_t*, int,
                              int64_t, int64_t, const moe_attn_params&, const moe_heads&, float*, void*, hipStream_t);
size_t attn_prompt_ws_bytes(int64_t, int64_t, int64_t, const moe_attn_params&);
size_t attn_decode_ws_bytes(int64_t, int, int, int, int, int64_t, int64_t);
int64_t attn_decode_grid(int64_t, int, int, int, int, int64_t, int64_t);
moe_status launch_attn_decode(const moe_heads&, const moe_kv_cache&, const int32_t*, int64_t, const int32_t*, int64_t,
                              int64_t, const int32_t*, int64_t, const moe_attn_params&, const moe_heads&, float*, void*,
                              hipStream_t);

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_kv_slots(const int32_t* cached_lens, const int32_t* new_lens, int32_t num_requests,
                        const int32_t* free_pages, int64_t num_free, int32_t page_size, int32_t* block_table,
                        int64_t table_stride, int32_t max_blocks, int32_t position_base, int64_t max_new, int32_t* slots,
                        int32_t* positions, int32_t* cu_new, int32_t* counts, hipStream_t stream) {
  set_error("");
  MOE_CHECK(num_requests >= 0 && num_free >= 0 && max_new >= 0 && position_base >= 0, "moe_kv_slots: negative size");
  if (num_requests > kv_slots_max_requests()) {
    set_error("moe_kv_slots: %d requests, at most %d", num_requests, kv_slots_max_requests());
    return MOE_ERR_UNSUPPORTED;
  }
  MOE_CHECK(is_pow2_int(page_size) && page_size <= 1024, "moe_kv_slots: page_size %d is no power of two up to 1024",
            page_size);
  MOE_CHECK(max_blocks >= 1 && (int64_t)max_blocks * page_size <= 0x7fffffff && table_stride >= max_blocks,
            "moe_kv_slots: bad max_blocks / table_stride");
  MOE_CHECK(max_new <= 0x7fffffff, "moe_kv_slots: max_new over 2^31 - 1");
  MOE_CHECK(cu_new && counts && (max_new == 0 || (slots && positions)), "moe_kv_slots: NULL output");
  MOE_CHECK(num_requests == 0 || (cached_lens && new_lens && block_table), "moe_kv_slots: NULL pointer");
  MOE_CHECK(num_free == 0 || free_pages, "moe_kv_slots: free_pages is NULL");
  return launch_kv_slots(cached_lens, new_lens, num_requests, free_pages, num_free, __builtin_ctz((unsigned)page_size),
                         block_table, table_stride, max_blocks, position_base, max_new, slots, positions, cu_new, counts,
                         stream);
}

moe_status moe_qk_norm_rope(const moe_heads* q, const moe_heads* k, const moe_heads* v, int64_t T,
                            const moe_rope_params* p, const int32_t* positions, const float* cos_sin,
                            const float* q_weight, const float* k_weight, const moe_heads* q_out, const moe_heads* k_out,
                            const moe_kv_cache* cache, const int32_t* slots, hipStream_t stream) {
  const char* fn = "moe_qk_norm_rope";
  set_error("");
  MOE_PASS(check_rope(fn, T, p));
  if (T == 0) return MOE_OK;
  MOE_PASS(check_rope_data(fn, T, p, q, k, positions, cos_sin, q_weight, k_weight, q_out, k_out));
  if (cache) {
    MOE_PASS(check_cache(fn, cache));
    MOE_CHECK(slots, "%s: a cache needs slots", fn);
    MOE_CHECK(p->v_dim >= 8 && p->v_dim % 8 == 0, "%s: v_dim %d is no positive multiple of 8", fn, p->v_dim);
    MOE_PASS(check_heads(fn, "v", v, p->kv_heads, p->v_dim, 0));
  } else {
    MOE_CHECK(k_out, "%s: keys go nowhere (neither k_out nor a cache)", fn);
  }
  MOE_CHECK(T * (p->q_heads + 2 * (int64_t)p->kv_heads) < ((int64_t)1 << 31), "%s: too many heads", fn);
  return launch_qk_norm_rope(*q, *k, v, T, *p, positions, cos_sin, q_weight, k_weight, *q_out, k_out, cache, slots,
                             stream);
}

size_t moe_attn_prompt_workspace_bytes(int32_t num_seqs, int64_t total_q, int64_t total_k, const moe_attn_params* p) {
  if (!sizes_of_heads(p) || num_seqs <= 0 || total_q <= 0 || total_k <= 0 || total_q > 0x7fffffff || total_k > 0x7fffffff) return 0;
  return attn_prompt_ws_bytes(total_q, total_k, num_seqs, *p);
}

moe_status moe_attn_prompt(const moe_heads* q, const moe_heads* k, const moe_heads* v, const int32_t* cu_q,
                           const int32_t* cu_k, int32_t num_seqs, int64_t total_q, int64_t total_k,
                           const moe_attn_params* p, const moe_heads* out, float* lse, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "moe_attn_prompt";
  set_error("");
  MOE_PASS(check_attn(fn, p));
  MOE_CHECK(num_seqs >= 0 && total_q >= 0 && total_k >= 0, "%s: negative size", fn);
  MOE_CHECK(total_q <= 0x7fffffff && total_k <= 0x7fffffff, "%s: over 2^31 - 1 rows", fn);
  if (num_seqs == 0 || total_q == 0) return MOE_OK;
  MOE_CHECK(cu_q && cu_k, "%s: cu_q / cu_k is NULL", fn);
  MOE_PASS(check_heads(fn, "q", q, p->q_heads, p->k_dim, 0));
  if (total_k > 0) {
    MOE_PASS(check_heads(fn, "k", k, p->kv_heads, p->k_dim, 0));
    MOE_PASS(check_heads(fn, "v", v, p->kv_heads, p->v_dim, 0));
  }
  MOE_PASS(check_heads(fn, "out", out, p->q_heads, p->v_dim, total_q));
  MOE_CHECK(aligned4(lse), "%s: lse not 4-byte aligned", fn);
  // a tile of 64 rows is addressed with 31 bits
  if (total_k > 0 && (k->token_stride > (1 << 23) || v->token_stride > (1 << 23))) {
    set_error("%s: token strides of k and v over 2^23 elements are not supported", fn);
    return MOE_ERR_UNSUPPORTED;
  }
  // rows (queries x heads of a key head), their tiles and the grid in 31 bits
  MOE_CHECK(total_q * (p->q_heads / p->kv_heads) <= 0x7fffffff - 1024 - num_seqs &&
                (total_q * p->q_heads / 128 + (int64_t)num_seqs * p->kv_heads) < ((int64_t)1 << 31),
            "%s: too many rows", fn);
  const size_t need = attn_prompt_ws_bytes(total_q, total_k, num_seqs, *p);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))) {
    set_error("%s: workspace %zu bytes < %zu (or NULL / unaligned)", fn, workspace_bytes, need);
    return MOE_ERR_WORKSPACE;
  }
  static const moe_heads none = {nullptr, 0, 0};
  return launch_attn_prompt(*q, total_k > 0 ? *k : none, total_k > 0 ? *v : none, cu_q, cu_k, num_seqs, total_q, total_k,
                            *p, *out, lse, workspace, stream);
}

size_t moe_attn_decode_workspace_bytes(int32_t num_requests, int64_t prefix_len, int64_t max_len,
                                       const moe_attn_params* p) {
  if (!sizes_of_heads(p) || num_requests <= 0 || prefix_len < 0 || max_len < 0 ||
      !decode_sizes_fit(num_requests, prefix_len, max_len, *p))
    return 0;
  return attn_decode_ws_bytes(num_requests, p->q_heads, p->kv_heads, p->k_dim, p->v_dim, prefix_len, max_len);
}

moe_status moe_attn_decode(const moe_heads* q, const moe_kv_cache* cache, const int32_t* block_table,
                           int64_t table_stride, int32_t max_blocks, const int32_t* lens, int32_t num_requests,
                           int64_t max_len, const int32_t* prefix_table, int32_t prefix_blocks, int64_t prefix_len,
                           const moe_attn_params* p, const moe_heads* out, float* lse, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "moe_attn_decode";
  set_error("");
  MOE_PASS(check_attn(fn, p));
  MOE_CHECK(num_requests >= 0 && max_len >= 0 && prefix_len >= 0 && max_blocks >= 0 && prefix_blocks >= 0,
            "%s: negative size", fn);
  if (num_requests == 0) return MOE_OK;
  MOE_PASS(check_cache(fn, cache));
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
  MOE_CHECK(attn_decode_grid(num_requests, p->q_heads, p->kv_heads, p->k_dim, p->v_dim, prefix_len, max_len) < ((int64_t)1 << 31),
            "%s: too many rows", fn);
  const size_t need = attn_decode_ws_bytes(num_requests, p->q_heads, p->kv_heads, p->k_dim, p->v_dim, prefix_len, max_len);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))) {
    set_error("%s: workspace %zu bytes < %zu (or NULL / unaligned)", fn, workspace_bytes, need);
    return MOE_ERR_WORKSPACE;
  }
  return launch_attn_decode(*q, *cache, block_table, table_stride, lens, num_requests, max_len, prefix_table, prefix_len,
                            *p, *out, lse, workspace, stream);
}

}  // extern "C"
