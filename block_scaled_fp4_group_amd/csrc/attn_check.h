// Argument checks shared by the entry points of the attention calls and of the calls
// around their cache.
#pragma once
#include <cmath>

#include "abi_check.h"

#define MOE_PASS(call)                 \
  do {                                 \
    const moe_status pass_st = (call); \
    if (pass_st != MOE_OK) return pass_st; \
  } while (0)

namespace moe {

inline bool is_pow2_int(int32_t x) { return x > 0 && (x & (x - 1)) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// rows of `heads` heads of `dim` bf16 each: 16-byte loads and stores
// (out_tokens > 0: the rows are written and must not overlap, in either order of tokens and heads)
inline moe_status check_heads(const char* fn, const char* name, const moe_heads* x, int32_t heads, int32_t dim,
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

inline moe_status check_cache(const char* fn, const moe_kv_cache* c) {
  MOE_CHECK(c && c->k && c->v, "%s: cache is NULL", fn);
  MOE_CHECK(aligned16(c->k) && aligned16(c->v), "%s: cache must be 16-byte aligned", fn);
  MOE_CHECK(is_pow2_int(c->page_size) && c->page_size <= 1024, "%s: page_size %d is no power of two up to 1024", fn,
            c->page_size);
  MOE_CHECK(c->num_pages >= 1 && c->num_pages <= (int64_t)0x7fffffff / c->page_size,
            "%s: num_pages outside [1, 2^31 / page_size)", fn);
  return MOE_OK;
}

inline moe_status check_attn(const char* fn, const moe_attn_params* p) {
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

// sizes of the head norms and the rotation
inline moe_status check_rope(const char* fn, int64_t T, const moe_rope_params* p) {
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
  return MOE_OK;
}

// what they read and write besides a cache (T > 0)
inline moe_status check_rope_data(const char* fn, int64_t T, const moe_rope_params* p, const moe_heads* q, const moe_heads* k,
                                  const int32_t* positions, const float* cos_sin, const float* q_weight,
                                  const float* k_weight, const moe_heads* q_out, const moe_heads* k_out) {
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
  return MOE_OK;
}

// what both workspace queries need of the parameters
inline bool sizes_of_heads(const moe_attn_params* p) {
  return p && p->kv_heads >= 1 && p->q_heads >= p->kv_heads && p->q_heads <= 65536 && p->q_heads % p->kv_heads == 0 &&
         p->k_dim >= 1 && p->k_dim <= 1024 && p->v_dim >= 1 && p->v_dim <= 1024;
}

// a launch's threads are counted in 32 bits
inline bool launch_fits(int64_t workgroups, int64_t threads) { return workgroups * threads < ((int64_t)1 << 32); }

// sizes that a plan is made for: rows and keys in 31 bits
inline bool decode_sizes_fit(int32_t num_requests, int64_t prefix_len, int64_t max_len, const moe_attn_params& p) {
  return max_len <= 0x7fffffff - 64 && prefix_len <= 0x7fffffff - 64 && num_requests * ((max_len + 31) / 32) < 0x7fffffff &&
         (int64_t)num_requests * p.q_heads < ((int64_t)1 << 31);
}

}  // namespace moe
