// C entry points of the attention operators: argument checks, then launches.
#include <cmath>

#include "abi_check.h"

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

static bool is_pow2_int(int32_t x) { return x > 0 && (x & (x - 1)) == 0; }
static bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// rows of `heads` heads of `dim` bf16 each: 16-byte loads and stores
// (out_tokens > 0: the rows are written and must not overlap, in either order of tokens and heads)
static moe_status check_heads(const char* fn, const char* name, const moe_heads* x, int32_t heads, int32_t dim,
                              int64_t out_tokens) {
  MOE_CHECK(x && x->data, "%s: %s is NULL", fn, name);
  MOE_CHECK(aligned16(x->data) && x->token_stride % 8 == 0 && x->head_stride % 8 == 0,
            "%s: %s needs 16-byte alignment and strides that are multiples of 8 elements", fn, name);
  MOE_CHECK(x->token_stride >= 0 && x->head_stride >= 0, "%s: %s has a negative stride", fn, name);
  if (out_tokens > 0) {
    const int64_t ts = x->token_stride, hs = x->head_stride;
    auto apart = [&](int64_t inner, int64_t n, int64_t outer, int64_t m) {
      return (n == 1 || inner >= dim) && (m == 1 || outer >= (n - 1) * inner + dim);
    };
    MOE_CHECK(apart(hs, heads, ts, out_tokens) || apart(ts, out_tokens, hs, heads), "%s: rows of %s overlap", fn, name);
  }
  return MOE_OK;
}

static moe_status check_cache(const char* fn, const moe_kv_cache* c) {
  MOE_CHECK(c && c->k && c->v, "%s: cache is NULL", fn);
  MOE_CHECK(aligned16(c->k) && aligned16(c->v), "%s: cache must be 16-byte aligned", fn);
  MOE_CHECK(is_pow2_int(c->page_size) && c->page_size <= 1024, "%s: page_size %d is no power of two up to 1024", fn,
            c->page_size);
  MOE_CHECK(c->num_pages >= 1 && c->num_pages <= (int64_t)0x7fffffff / c->page_size,
            "%s: num_pages outside [1, 2^31 / page_size)", fn);
  return MOE_OK;
}

static moe_status check_attn(const char* fn, const moe_attn_params* p) {
  MOE_CHECK(p, "%s: params is NULL", fn);
  MOE_CHECK(p->kv_heads >= 1 && p->q_heads >= p->kv_heads && p->q_heads % p->kv_heads == 0 && p->q_heads <= 65536,
            "%s: q_heads %d is no multiple of kv_heads %d", fn, p->q_heads, p->kv_heads);
  MOE_CHECK(p->scale > 0.0f && std::isfinite(p->scale), "%s: scale must be positive and finite", fn);
  const bool known = (p->k_dim == 64 && p->v_dim == 64) || (p->k_dim == 128 && p->v_dim == 128) ||
                     (p->k_dim == 192 && p->v_dim == 128);
  if (!known) {
    set_error("%s: head sizes (keys %d, values %d) are not built; (64, 64), (128, 128) and (192, 128) are", fn, p->k_dim,
              p->v_dim);
    return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

#define MOE_PASS(call)                 \
  do {                                 \
    const moe_status pass_st = (call); \
    if (pass_st != MOE_OK) return pass_st; \
  } while (0)

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
  MOE_CHECK(p, "%s: params is NULL", fn);
  MOE_CHECK(T >= 0 && T <= 0x7fffffff && p->q_heads >= 1 && p->kv_heads >= 1 && p->q_heads <= 65536 && p->kv_heads <= 65536,
            "%s: bad sizes", fn);
  MOE_CHECK(p->eps >= 0.0f && std::isfinite(p->eps), "%s: eps must be finite and not negative", fn);
  MOE_CHECK(p->rot_dim >= 0 && p->rot_dim <= p->head_dim && p->rot_dim % 16 == 0,
            "%s: rot_dim %d is no multiple of 16 up to head_dim", fn, p->rot_dim);
  if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 192) {
    set_error("%s: head_dim %d is not built; 64, 128 and 192 are", fn, p->head_dim);
    return MOE_ERR_UNSUPPORTED;
  }
  if (T == 0) return MOE_OK;
  MOE_PASS(check_heads(fn, "q", q, p->q_heads, p->head_dim, 0));
  MOE_PASS(check_heads(fn, "k", k, p->kv_heads, p->head_dim, 0));
  MOE_PASS(check_heads(fn, "q_out", q_out, p->q_heads, p->head_dim, T));
  if (k_out) MOE_PASS(check_heads(fn, "k_out", k_out, p->kv_heads, p->head_dim, T));
  if (p->rot_dim > 0) {
    MOE_CHECK(positions && cos_sin && p->max_position >= 1, "%s: rotation needs positions and a cos / sin table", fn);
    MOE_CHECK(aligned16(cos_sin), "%s: cos_sin must be 16-byte aligned", fn);
  }
  MOE_CHECK((!q_weight || aligned16(q_weight)) && (!k_weight || aligned16(k_weight)),
            "%s: weights must be 16-byte aligned", fn);
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

// what both workspace queries need of the parameters
static bool sizes_of_heads(const moe_attn_params* p) {
  return p && p->kv_heads >= 1 && p->q_heads >= p->kv_heads && p->q_heads <= 65536 && p->q_heads % p->kv_heads == 0 &&
         p->k_dim >= 1 && p->k_dim <= 1024 && p->v_dim >= 1 && p->v_dim <= 1024;
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

// sizes that a plan is made for: rows and keys in 31 bits
static bool decode_sizes_fit(int32_t num_requests, int64_t prefix_len, int64_t max_len, const moe_attn_params& p) {
  return max_len <= 0x7fffffff - 64 && prefix_len <= 0x7fffffff - 64 && num_requests * ((max_len + 31) / 32) < 0x7fffffff &&
         (int64_t)num_requests * p.q_heads < ((int64_t)1 << 31);
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
