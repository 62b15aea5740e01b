// What the two forms of head norm + rotation + cache write share: a bf16 cache
// (qk_norm_rope.hip) and one held in 4 bits (qk_norm_rope_fp4.hip).
#pragma once
#include "common.h"

namespace moe {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  uint16_t* k_out;
  uint16_t* k_cache;
  uint16_t* v_cache;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
  const int32_t* positions;
  const int32_t* slots;
  const float* cos_sin;
  const float* q_weight;
  const float* k_weight;
  int64_t T, num_slots;
  int32_t q_heads, kv_heads, v_dim, rot, max_position;
  float eps;
};

__device__ __forceinline__ void unpack8(const u32x4& w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  return u32x4{cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]), cvt_bf16x2(x[6], x[7])};
}

// n floats from a 16-byte aligned address
template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f32x4 v = *(const f32x4*)(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i + j] = v[j];
  }
}

template <bool ONCE>
__device__ __forceinline__ void store8(uint16_t* p, u32x4 v) {
  if (ONCE) __builtin_nontemporal_store(v, (u32x4*)p);
  else *(u32x4*)p = v;
}

inline RopeArgs rope_args(const moe_heads& q, const moe_heads& k, const moe_heads* v, int64_t T, const moe_rope_params& p,
                          const int32_t* positions, const float* cos_sin, const float* q_weight, const float* k_weight,
                          const moe_heads& q_out, const moe_heads* k_out, const int32_t* slots) {
  RopeArgs a = {};
  a.q = (const uint16_t*)q.data;
  a.q_ts = q.token_stride;
  a.q_hs = q.head_stride;
  a.k = (const uint16_t*)k.data;
  a.k_ts = k.token_stride;
  a.k_hs = k.head_stride;
  a.v = v ? (const uint16_t*)v->data : nullptr;
  a.v_ts = v ? v->token_stride : 0;
  a.v_hs = v ? v->head_stride : 0;
  a.q_out = (uint16_t*)q_out.data;
  a.qo_ts = q_out.token_stride;
  a.qo_hs = q_out.head_stride;
  a.k_out = k_out ? (uint16_t*)k_out->data : nullptr;
  a.ko_ts = k_out ? k_out->token_stride : 0;
  a.ko_hs = k_out ? k_out->head_stride : 0;
  a.positions = positions;
  a.slots = slots;
  a.cos_sin = cos_sin;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.T = T;
  a.q_heads = p.q_heads;
  a.kv_heads = p.kv_heads;
  a.v_dim = p.v_dim;
  a.rot = p.rot_dim;
  a.max_position = p.max_position;
  a.eps = p.eps;
  return a;
}

}  // namespace moe
