// RMS norm of every query and key head, the position rotation and the cache
// write in one pass over the projection's output:
//   y = x * rsqrt(mean(x^2) + eps) * w              (per head; no weight: y = x)
//   pair i of the first rot_dim elements turned by the position's angle:
//   (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i)
// with pairs (i, i + rot_dim / 2) or, interleaved, (2 i, 2 i + 1).  Keys and
// values also go to their cache rows.  Everything is float until the one
// rounding to bf16 of each output.
//
// Memory traffic is all there is (a few operations per value).  A lane owns the
// 8 elements at e and the 8 at e + half of the rotated part (or of the rest), so
// both members of every pair of either kind sit in one lane, loads and stores
// are 16 bytes, and only the sum of squares crosses lanes.
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

// LPH lanes per head (a power of two >= D / 16); head h of token t: query heads
// first, then key heads, then (with a cache) value heads, which are copied
template <int D, bool INTERLEAVED>
__global__ __launch_bounds__(kRopeThreads) void qk_norm_rope_kernel(RopeArgs a) {
  constexpr int kLanes = D / 16;                                   // lanes with data
  constexpr int LPH = kLanes <= 4 ? 4 : (kLanes <= 8 ? 8 : 16);
  const int sub = threadIdx.x % LPH;
  const int64_t heads = a.q_heads + a.kv_heads + (a.v_cache ? a.kv_heads : 0);
  const int64_t item = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / LPH;
  if (item >= a.T * heads) return;                                 // whole groups of LPH lanes
  const int64_t t = item / heads;
  const int h = (int)(item - t * heads);
  const int64_t slot = a.slots ? a.slots[t] : -1;
  const bool cached = slot >= 0 && slot < a.num_slots;
  if (h >= a.q_heads + a.kv_heads) {
    const int hv = h - a.q_heads - a.kv_heads;
    if (!cached) return;
    const uint16_t* src = a.v + t * a.v_ts + hv * a.v_hs;
    uint16_t* dst = a.v_cache + (slot * a.kv_heads + hv) * a.v_dim;
    for (int e = sub * 8; e < a.v_dim; e += LPH * 8) *(u32x4*)(dst + e) = *(const u32x4*)(src + e);
    return;
  }
  const bool is_q = h < a.q_heads;
  const int hh = is_q ? h : h - a.q_heads;
  const uint16_t* src = is_q ? a.q + t * a.q_ts + hh * a.q_hs : a.k + t * a.k_ts + hh * a.k_hs;
  const float* w = is_q ? a.q_weight : a.k_weight;
  // lanes below rot / 16 hold rotated pairs, the others the rest; e, e + half
  const int nrot = a.rot / 16;
  const bool rotated = sub < nrot, active = sub < kLanes;
  const int half = rotated ? a.rot / 2 : (D - a.rot) / 2;
  const int e = active ? (rotated ? sub * 8 : a.rot + (sub - nrot) * 8) : 0;
  float x[8], y[8];
  if (active) {
    unpack8(*(const u32x4*)(src + e), x);
    unpack8(*(const u32x4*)(src + e + half), y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.0f;
  }
  if (w) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
    for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor(ss, d, LPH);
    const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
    if (active) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = x[i] * r * w[e + i];
        y[i] = y[i] * r * w[e + half + i];
      }
    }
  }
  if (!active) return;
  if (rotated) {
    const int64_t pos = min(max(a.positions[t], 0), a.max_position - 1);
    const float* cs = a.cos_sin + pos * a.rot;
    const int hr = a.rot / 2;
    if (INTERLEAVED) {
      auto turn = [&](float (&z)[8], int e0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = cs[e0 / 2 + i], s = cs[hr + e0 / 2 + i];
          const float p = z[2 * i], q = z[2 * i + 1];
          z[2 * i] = p * c - q * s;
          z[2 * i + 1] = q * c + p * s;
        }
      };
      turn(x, e);
      turn(y, e + half);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = cs[e + i], s = cs[hr + e + i];
        const float p = x[i], q = y[i];
        x[i] = p * c - q * s;
        y[i] = q * c + p * s;
      }
    }
  }
  const u32x4 o0 = pack8(x), o1 = pack8(y);
  uint16_t* dst = is_q ? a.q_out + t * a.qo_ts + hh * a.qo_hs
                       : (a.k_out ? a.k_out + t * a.ko_ts + hh * a.ko_hs : nullptr);
  if (dst) {
    *(u32x4*)(dst + e) = o0;
    *(u32x4*)(dst + e + half) = o1;
  }
  if (!is_q && a.k_cache && cached) {
    uint16_t* kc = a.k_cache + (slot * a.kv_heads + hh) * D;
    *(u32x4*)(kc + e) = o0;
    *(u32x4*)(kc + e + half) = o1;
  }
}

template <int D>
static void launch_rope_d(const RopeArgs& a, bool interleaved, hipStream_t stream) {
  constexpr int kLanes = D / 16;
  constexpr int LPH = kLanes <= 4 ? 4 : (kLanes <= 8 ? 8 : 16);
  const int64_t heads = a.q_heads + a.kv_heads + (a.v_cache ? a.kv_heads : 0);
  const int64_t per = kRopeThreads / LPH;
  const dim3 grid((uint32_t)((a.T * heads + per - 1) / per));
  if (interleaved)
    hipLaunchKernelGGL((qk_norm_rope_kernel<D, true>), grid, dim3(kRopeThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<D, false>), grid, dim3(kRopeThreads), 0, stream, a);
}

moe_status launch_qk_norm_rope(const moe_heads& q, const moe_heads& k, const moe_heads* v, int64_t T,
                               const moe_rope_params& p, const int32_t* positions, const float* cos_sin,
                               const float* q_weight, const float* k_weight, const moe_heads& q_out,
                               const moe_heads* k_out, const moe_kv_cache* cache, const int32_t* slots,
                               hipStream_t stream) {
  RopeArgs a;
  a.q = (const uint16_t*)q.data;
  a.q_ts = q.token_stride;
  a.q_hs = q.head_stride;
  a.k = (const uint16_t*)k.data;
  a.k_ts = k.token_stride;
  a.k_hs = k.head_stride;
  a.v = cache ? (const uint16_t*)v->data : nullptr;
  a.v_ts = cache ? v->token_stride : 0;
  a.v_hs = cache ? v->head_stride : 0;
  a.q_out = (uint16_t*)q_out.data;
  a.qo_ts = q_out.token_stride;
  a.qo_hs = q_out.head_stride;
  a.k_out = k_out ? (uint16_t*)k_out->data : nullptr;
  a.ko_ts = k_out ? k_out->token_stride : 0;
  a.ko_hs = k_out ? k_out->head_stride : 0;
  a.k_cache = cache ? (uint16_t*)cache->k : nullptr;
  a.v_cache = cache ? (uint16_t*)cache->v : nullptr;
  a.num_slots = cache ? cache->num_pages * cache->page_size : 0;
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
  switch (p.head_dim) {
    case 64: launch_rope_d<64>(a, p.interleaved, stream); break;
    case 128: launch_rope_d<128>(a, p.interleaved, stream); break;
    default: launch_rope_d<192>(a, p.interleaved, stream); break;
  }
  return launch_status("moe_qk_norm_rope");
}

}  // namespace moe
