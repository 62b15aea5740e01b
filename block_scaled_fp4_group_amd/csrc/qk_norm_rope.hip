// RMS norm of every query and key head, the position rotation and the cache
// write in one pass over the projection's output:
//   y = x * rsqrt(mean(x^2) + eps) * w              (per head; no weight: y = x)
//   pair i of the first rot_dim elements turned by the position's angle:
//   (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i)
// with pairs (i, i + rot_dim / 2) or, interleaved, (2 i, 2 i + 1).  Keys and
// values also go to their cache rows.  Everything is float until the one
// rounding to bf16 of each output.
//
// Memory traffic is all there is (a few operations per value): 8191 tokens x 64/4
// heads x 192 read and write 459 MB in 96 us, 4.8 TB/s where a large copy reaches
// 5.1; 64 tokens x 32/8 x 128 take 3.5 us, a launch's latency.  A lane owns the
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
  // a cache held in 4 bits
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  int32_t page_shift;
  float k_inv, v_inv;                               // 1 / global scale, a power of two
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

// ------------------------------------------------- a cache held in 4 bits
// NVFP4: 16 values to a block, which is what two neighbouring lanes hold (8 each).
// Scale: E4M3 of the block's largest magnitude / 6; codes: E2M1 of value / scale; both to
// the nearest, ties to even.  Page p of head h is [page_size] rows of codes and, for keys,
// of scales; the values' scales are [v_dim / 16][page_size], as the attention call
// reads a block's scales of many keys at once.

// E4M3 byte of v >= 0, saturating at 448.
__device__ __forceinline__ uint32_t f64_to_e4m3_sat(double v) {
  if (!(v > 0.0)) return 0u;
  if (v >= 448.0) return 0x7Eu;
  const int e = max((int)((__double_as_longlong(v) >> 52) & 0x7ff) - 1023, -6);
  // steps of 2^(e - 3); 8 to 16 of them above 2^-6, where 16 carries into the exponent
  const int n = (int)rint(v * __longlong_as_double((int64_t)(1023 + 3 - e) << 52));
  return (uint32_t)(e == -6 ? n : ((e + 7) << 3) + n - 8);
}

// Codes of this lane's 8 values of a block (value i in nibble i) and the block's scale byte.
// In double: a value next to the border between two codes lands on its own side of it.
// Keys come out of norm and rotation in double too: in float about one code in 10^6 is its
// neighbour.
__device__ __forceinline__ uint32_t fp4_block(const double (&x)[8], double inv_global, uint32_t* scale) {
  double most = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmax(most, fabs(x[i]));
  most = fmax(most, __shfl_xor(most, 1));
  *scale = f64_to_e4m3_sat(most * inv_global / 6.0);
  const double s = (double)e4m3_to_f32(*scale);
  if (s == 0.0) return 0u;
  uint32_t w = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double a = fabs(x[i]) * inv_global;                       // exact, as the borders are
    uint32_t c = (a > 0.25 * s) + (a >= 0.75 * s) + (a > 1.25 * s) + (a >= 1.75 * s) + (a > 2.5 * s) + (a >= 3.5 * s) +
                 (a > 5.0 * s);
    c |= signbit(x[i]) ? 8u : 0u;
    w |= c << (4 * i);
  }
  return w;
}

// LPH lanes per head (a power of two >= D / 16); head h of token t: query heads
// first, then key heads, then (with a cache) value heads, which are copied.
// FAR: outputs stored non-temporally.  FP4: the cache is held in 4 bits; keys are then
// computed in double.
template <int D, bool INTERLEAVED, bool FAR, bool FP4>
__global__ __launch_bounds__(kRopeThreads) void qk_norm_rope_kernel(RopeArgs a) {
  constexpr int kLanes = D / 16;                                   // lanes with data
  constexpr int LPH = kLanes <= 4 ? 4 : (kLanes <= 8 ? 8 : 16);
  const int sub = threadIdx.x % LPH;
  const uint32_t heads = (uint32_t)(a.q_heads + a.kv_heads + (a.v ? a.kv_heads : 0));
  const uint32_t item = blockIdx.x * (uint32_t)(kRopeThreads / LPH) + threadIdx.x / LPH;
  if (item >= (uint32_t)a.T * heads) return;                       // whole groups of LPH lanes; < 2^31 (host)
  const int64_t t = item / heads;
  const int h = (int)(item % heads);
  const int64_t slot = a.slots ? a.slots[t] : -1;
  const bool cached = slot >= 0 && slot < a.num_slots;
  if (h >= a.q_heads + a.kv_heads) {
    const int hv = h - a.q_heads - a.kv_heads;
    if (!cached) return;
    const uint16_t* src = a.v + t * a.v_ts + hv * a.v_hs;
    if (FP4) {
      const int64_t page = slot >> a.page_shift, row = slot - (page << a.page_shift), head = page * a.kv_heads + hv;
      for (int e = sub * 8; e < a.v_dim; e += LPH * 8) {            // (a block's two lanes go on together)
        float x[8];
        double z[8];
        unpack8(*(const u32x4*)(src + e), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = x[i];
        uint32_t s;
        const uint32_t w = fp4_block(z, a.v_inv, &s);
        *(uint32_t*)(a.v_codes + ((head << a.page_shift) + row) * (a.v_dim / 2) + e / 2) = w;
        if ((sub & 1) == 0) a.v_scales[((head * (a.v_dim / 16) + e / 16) << a.page_shift) + row] = (uint8_t)s;
      }
      return;
    }
    uint16_t* dst = a.v_cache + (slot * a.kv_heads + hv) * a.v_dim;
    for (int e = sub * 8; e < a.v_dim; e += LPH * 8) store8<FAR>(dst + e, *(const u32x4*)(src + e));
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
  if (FP4 && !is_q) {
    // the same in double, then the block's codes; the lanes without data go along to the exchanges
    double xd[8], yd[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      xd[i] = x[i];
      yd[i] = y[i];
    }
    if (w) {
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fma(xd[i], xd[i], fma(yd[i], yd[i], ss));
#pragma unroll
      for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor(ss, d, LPH);
      const double r = 1.0 / sqrt(ss * (1.0 / D) + (double)a.eps);
      float wx[8], wy[8];
      load_f32(w + e, wx);
      load_f32(w + e + half, wy);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xd[i] = xd[i] * r * wx[i];
        yd[i] = yd[i] * r * wy[i];
      }
    }
    if (rotated) {
      const int64_t pos = min(max(a.positions[t], 0), a.max_position - 1);
      const float* cs = a.cos_sin + pos * a.rot;
      const int hr = a.rot / 2;
      if (INTERLEAVED) {
        auto turn = [&](double (&z)[8], int e0) {
          float c[4], s[4];
          load_f32(cs + e0 / 2, c);
          load_f32(cs + hr + e0 / 2, s);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const double p = z[2 * i], q = z[2 * i + 1];
            z[2 * i] = p * c[i] - q * s[i];
            z[2 * i + 1] = q * c[i] + p * s[i];
          }
        };
        turn(xd, e);
        turn(yd, e + half);
      } else {
        float c[8], s[8];
        load_f32(cs + e, c);
        load_f32(cs + hr + e, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double p = xd[i], q = yd[i];
          xd[i] = p * c[i] - q * s[i];
          yd[i] = q * c[i] + p * s[i];
        }
      }
    }
    uint32_t s0, s1;
    const uint32_t w0 = fp4_block(xd, a.k_inv, &s0), w1 = fp4_block(yd, a.k_inv, &s1);
    if (!active) return;
    if (a.k_out) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = (float)xd[i];
        y[i] = (float)yd[i];
      }
      uint16_t* dst = a.k_out + t * a.ko_ts + hh * a.ko_hs;
      store8<FAR>(dst + e, pack8(x));
      store8<FAR>(dst + e + half, pack8(y));
    }
    if (cached) {
      const int64_t page = slot >> a.page_shift, row = slot - (page << a.page_shift);
      const int64_t at = ((page * a.kv_heads + hh) << a.page_shift) + row;
      *(uint32_t*)(a.k_codes + at * (D / 2) + e / 2) = w0;
      *(uint32_t*)(a.k_codes + at * (D / 2) + (e + half) / 2) = w1;
      if ((sub & 1) == 0) {
        a.k_scales[at * (D / 16) + e / 16] = (uint8_t)s0;
        a.k_scales[at * (D / 16) + (e + half) / 16] = (uint8_t)s1;
      }
    }
    return;
  }
  if (w) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
    for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor(ss, d, LPH);
    const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
    float wx[8], wy[8];
    load_f32(w + e, wx);
    load_f32(w + e + half, wy);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = x[i] * r * wx[i];
      y[i] = y[i] * r * wy[i];
    }
  }
  if (!active) return;
  if (rotated) {
    const int64_t pos = min(max(a.positions[t], 0), a.max_position - 1);
    const float* cs = a.cos_sin + pos * a.rot;
    const int hr = a.rot / 2;
    if (INTERLEAVED) {
      auto turn = [&](float (&z)[8], int e0) {
        float c[4], s[4];
        load_f32(cs + e0 / 2, c);
        load_f32(cs + hr + e0 / 2, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = z[2 * i], q = z[2 * i + 1];
          z[2 * i] = p * c[i] - q * s[i];
          z[2 * i + 1] = q * c[i] + p * s[i];
        }
      };
      turn(x, e);
      turn(y, e + half);
    } else {
      float c[8], s[8];
      load_f32(cs + e, c);
      load_f32(cs + hr + e, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = x[i], q = y[i];
        x[i] = p * c[i] - q * s[i];
        y[i] = q * c[i] + p * s[i];
      }
    }
  }
  const u32x4 o0 = pack8(x), o1 = pack8(y);
  uint16_t* dst = is_q ? a.q_out + t * a.qo_ts + hh * a.qo_hs
                       : (a.k_out ? a.k_out + t * a.ko_ts + hh * a.ko_hs : nullptr);
  if (dst) {
    store8<FAR>(dst + e, o0);
    store8<FAR>(dst + e + half, o1);
  }
  if (!FP4 && !is_q && a.k_cache && cached) {
    uint16_t* kc = a.k_cache + (slot * a.kv_heads + hh) * D;
    store8<FAR>(kc + e, o0);
    store8<FAR>(kc + e + half, o1);
  }
}

// Outputs larger than half of the 256 MB cache before HBM are not there any more
// when the next kernel reads them, and go out non-temporally: 8191 x 64/4 x 192
// (230 MB) 100 -> 96 us, 4.8 TB/s read and written where a copy reaches 5.1.
// Smaller ones stay for their reader.
template <int D, bool INTERLEAVED, bool FP4>
static void launch_rope_d(const RopeArgs& a, hipStream_t stream) {
  constexpr int kLanes = D / 16;
  constexpr int LPH = kLanes <= 4 ? 4 : (kLanes <= 8 ? 8 : 16);
  const int64_t heads = a.q_heads + a.kv_heads + (a.v ? a.kv_heads : 0);
  const int64_t per = kRopeThreads / LPH;
  const dim3 grid((uint32_t)((a.T * heads + per - 1) / per));
  if (a.T * heads * D * 2 > ((int64_t)128 << 20))
    hipLaunchKernelGGL((qk_norm_rope_kernel<D, INTERLEAVED, true, FP4>), grid, dim3(kRopeThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<D, INTERLEAVED, false, FP4>), grid, dim3(kRopeThreads), 0, stream, a);
}

template <bool FP4>
static void launch_rope(const RopeArgs& a, int D, bool interleaved, hipStream_t stream) {
  switch (D) {
    case 64: interleaved ? launch_rope_d<64, true, FP4>(a, stream) : launch_rope_d<64, false, FP4>(a, stream); break;
    case 128: interleaved ? launch_rope_d<128, true, FP4>(a, stream) : launch_rope_d<128, false, FP4>(a, stream); break;
    default: interleaved ? launch_rope_d<192, true, FP4>(a, stream) : launch_rope_d<192, false, FP4>(a, stream); break;
  }
}

static RopeArgs rope_args(const moe_heads& q, const moe_heads& k, const moe_heads* v, int64_t T, const moe_rope_params& p,
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

moe_status launch_qk_norm_rope(const moe_heads& q, const moe_heads& k, const moe_heads* v, int64_t T,
                               const moe_rope_params& p, const int32_t* positions, const float* cos_sin,
                               const float* q_weight, const float* k_weight, const moe_heads& q_out,
                               const moe_heads* k_out, const moe_kv_cache* cache, const int32_t* slots,
                               hipStream_t stream) {
  RopeArgs a = rope_args(q, k, cache ? v : nullptr, T, p, positions, cos_sin, q_weight, k_weight, q_out, k_out, slots);
  a.k_cache = cache ? (uint16_t*)cache->k : nullptr;
  a.v_cache = cache ? (uint16_t*)cache->v : nullptr;
  a.num_slots = cache ? cache->num_pages * cache->page_size : 0;
  launch_rope<false>(a, p.head_dim, p.interleaved, stream);
  return launch_status("moe_qk_norm_rope");
}

moe_status launch_qk_norm_rope_fp4(const moe_heads& q, const moe_heads& k, const moe_heads& v, int64_t T,
                                   const moe_rope_params& p, const int32_t* positions, const float* cos_sin,
                                   const float* q_weight, const float* k_weight, const moe_heads& q_out,
                                   const moe_heads* k_out, const moe_kv_cache_fp4& cache, const int32_t* slots,
                                   hipStream_t stream) {
  RopeArgs a = rope_args(q, k, &v, T, p, positions, cos_sin, q_weight, k_weight, q_out, k_out, slots);
  a.k_codes = (uint8_t*)cache.k;
  a.k_scales = (uint8_t*)cache.k_scale;
  a.v_codes = (uint8_t*)cache.v;
  a.v_scales = (uint8_t*)cache.v_scale;
  a.num_slots = cache.num_pages * cache.page_size;
  a.page_shift = __builtin_ctz((unsigned)cache.page_size);
  a.k_inv = 1.0f / cache.k_global;
  a.v_inv = 1.0f / cache.v_global;
  launch_rope<true>(a, p.head_dim, p.interleaved, stream);
  return launch_status("moe_qk_norm_rope_fp4");
}

}  // namespace moe
