// RMS norm of every query and key head and the position rotation, as qk_norm_rope.hip,
// with keys and values quantised into a cache held in 4 bits.
//
// NVFP4: 16 values to a block, which is what two neighbouring lanes hold (8 each).
// Scale: E4M3 of the block's largest magnitude / 6; codes: E2M1 of value / scale; both to
// the nearest, ties to even.  Page p of head h is [page_size] rows of codes and, for keys,
// of scales; the values' scales are [v_dim / 16][page_size], as the attention call
// reads a block's scales of many keys at once.
//
// A lane owns the 8 elements at e and the 8 at e + half of the rotated part (or of the
// rest), as in the bf16 form.  Vector work would bound it there -- 336 instructions for 16
// values of a head, 94 us of 122 at 8191 tokens x 64/4 x 192 -- so a group of lanes takes
// four query heads of a token: addresses, weights, cosines and sines once, all heads' loads
// under way at once (122 -> 92 us, 4.8 TB/s where a large copy reaches 5.1; never slower than a
// head at a time from 64 tokens on).
#include "rope.h"

namespace moe {

// E4M3 byte of v >= 0, saturating at 448.
__device__ __forceinline__ uint32_t f64_to_e4m3_sat(double v) {
  if (!(v > 0.0)) return 0u;
  if (v >= 448.0) return 0x7Eu;
  const int e = max((int)((__double_as_longlong(v) >> 52) & 0x7ff) - 1023, -6);
  // steps of 2^(e - 3); 8 to 16 of them above 2^-6, where 16 carries into the exponent
  const int n = (int)rint(v * __longlong_as_double((int64_t)(1023 + 3 - e) << 52));
  return (uint32_t)(e == -6 ? n : ((e + 7) << 3) + n - 8);
}

// x as a float that lies to numbers of few bits as x does: cut off, the last bit set if
// anything was.
__device__ __forceinline__ float f64_to_odd(double x) {
  const float f = (float)x;
  const double d = (double)f;
  const uint32_t u = __float_as_uint(f) - (fabs(d) > fabs(x) ? 1u : 0u);
  return __uint_as_float(d == x ? u : u | 1u);
}

// A quotient by s from r = 1 / s, rounded once: the product's remainder put right (which
// takes the sign off a zero).
template <class F>
__device__ __forceinline__ F quotient(F a, F s, F r) {
  const F q = a * r;
  return copysign(fma(fma(-q, s, a), r, q), a);
}
// The quotients' E2M1 codes, to the nearest, ties to even, as bits 8 SEL .. 8 SEL + 7 of w.
template <int SEL>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w, float a, float b) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, 1.0f, SEL);
}
// Not a number counts as 0; past 8 s everything is 6 s.
__device__ __forceinline__ float in_reach(float a, float s) {
  const float most = 8.0f * s;
  return a == a ? fminf(fmaxf(a, -most), most) : copysignf(0.0f, a);
}
__device__ __forceinline__ double in_reach(double a, double s) {
  const double most = 8.0 * s;
  return a == a ? fmin(fmax(a, -most), most) : copysign(0.0, a);
}

// Codes of this lane's 8 values of a block (value i in nibble i) and the block's scale byte.
// Keys come out of norm and rotation in double: a value next to the border between two codes
// lands on its own side of it, where in float about one code in 10^6 is its neighbour.
__device__ __forceinline__ uint32_t fp4_block(const double (&x)[8], float inv_global, uint32_t* scale) {
  double most = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmax(most, fabs(x[i]));
  most = fmax(most, __shfl_xor(most, 1));
  *scale = f64_to_e4m3_sat(most * (double)inv_global / 6.0);
  const double s = (double)e4m3_to_f32(*scale);
  if (s == 0.0) return 0u;
  const double r = 1.0 / s;
  auto q = [&](int i) { return f64_to_odd(quotient(in_reach(x[i] * (double)inv_global, s), s, r)); };
  uint32_t w = e2m1_pair<0>(0u, q(0), q(1));
  __builtin_amdgcn_sched_barrier(0);                                // (few registers: reads wait to be issued)
  w = e2m1_pair<1>(w, q(2), q(3));
  __builtin_amdgcn_sched_barrier(0);
  w = e2m1_pair<2>(w, q(4), q(5));
  __builtin_amdgcn_sched_barrier(0);
  return e2m1_pair<3>(w, q(6), q(7));
}
// Values as they are: of bf16 values the quotients by scales of 4 bits are no nearer to a
// border than float tells, unless they lie on it.
__device__ __forceinline__ uint32_t fp4_block(const float (&x)[8], float inv_global, uint32_t* scale) {
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(x[i]));
  most = fmaxf(most, __shfl_xor(most, 1));
  *scale = f32_to_e4m3_sat(most * inv_global / 6.0f);
  const float s = e4m3_to_f32(*scale);
  if (s == 0.0f) return 0u;
  const float r = 1.0f / s;
  auto q = [&](int i) { return quotient(in_reach(x[i] * inv_global, s), s, r); };
  uint32_t w = e2m1_pair<0>(0u, q(0), q(1));
  w = e2m1_pair<1>(w, q(2), q(3));
  w = e2m1_pair<2>(w, q(4), q(5));
  return e2m1_pair<3>(w, q(6), q(7));
}

struct RopeFp4Args {
  RopeArgs r;
  uint8_t* k_codes;
  uint8_t* k_scales;
  uint8_t* v_codes;
  uint8_t* v_scales;
  int32_t page_shift;
  uint32_t tokens;
  float k_inv, v_inv;                               // 1 / global scale, a power of two
};

// A lane's part of the tables: weights of its elements (1 without), cosines and sines of its
// pairs -- (x[i], y[i]), or (x[2 i], x[2 i + 1]) and then (y[2 i], y[2 i + 1]) interleaved.
struct RopeTables {
  float wx[8], wy[8], c[8], s[8];
};
template <bool INTERLEAVED>
__device__ __forceinline__ void load_tables(const RopeArgs& a, const float* w, int64_t t, int e, int half, bool rotated,
                                            RopeTables* z) {
  if (w) {
    load_f32(w + e, z->wx);
    load_f32(w + e + half, z->wy);
  }
  if (!rotated) return;
  const float* cs = a.cos_sin + (int64_t)min(max(a.positions[t], 0), a.max_position - 1) * a.rot;
  const int hr = a.rot / 2;
  if (INTERLEAVED) {
    float u[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      load_f32(cs + (e + k * half) / 2, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) z->c[4 * k + i] = u[i];
      load_f32(cs + hr + (e + k * half) / 2, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) z->s[4 * k + i] = u[i];
    }
  } else {
    load_f32(cs + e, z->c);
    load_f32(cs + hr + e, z->s);
  }
}
__device__ __forceinline__ float inv_root(float x) { return 1.0f / sqrtf(x); }
__device__ __forceinline__ double inv_root(double x) { return 1.0 / sqrt(x); }

// Norm and rotation of the 16 elements that a lane holds of a head, its LPH lanes together.
template <int D, int LPH, bool INTERLEAVED, class F>
__device__ __forceinline__ void norm_rotate(const RopeTables& z, bool norm, float eps, bool rotated, F (&x)[8], F (&y)[8]) {
  if (norm) {
    F ss = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma(x[i], x[i], fma(y[i], y[i], ss));
#pragma unroll
    for (int d = 1; d < LPH; d <<= 1) ss += __shfl_xor(ss, d, LPH);
    const F r = inv_root(ss * ((F)1 / D) + (F)eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = x[i] * r * z.wx[i];
      y[i] = y[i] * r * z.wy[i];
    }
  }
  if (!rotated) return;
  auto turn = [](F& a, F& b, float c, float s) {
    const F p = a, q = b;
    a = p * c - q * s;
    b = q * c + p * s;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!INTERLEAVED) turn(x[i], y[i], z.c[i], z.s[i]);
    else if (i < 4) turn(x[2 * i], x[2 * i + 1], z.c[i], z.s[i]);
    else turn(y[2 * i - 8], y[2 * i - 7], z.c[i], z.s[i]);
  }
}

constexpr int QH = 4;

// LPH lanes per item (a power of two >= D / 16).  Items: of `tokens` tokens the query heads, QH
// of a token at a time, their key heads, their value heads, then the next.  FAR: outputs
// stored non-temporally.
template <int D, bool INTERLEAVED, bool FAR>
__global__ __launch_bounds__(kRopeThreads) void qk_norm_rope_fp4_kernel(RopeFp4Args p) {
  const RopeArgs& a = p.r;
  constexpr int kLanes = D / 16;                                   // lanes with data
  constexpr int LPH = kLanes <= 4 ? 4 : (kLanes <= 8 ? 8 : 16);
  const int sub = threadIdx.x % LPH;
  const uint32_t groups = (uint32_t)(a.q_heads + QH - 1) / QH, heads = (uint32_t)a.kv_heads;
  uint32_t item = blockIdx.x * (uint32_t)(kRopeThreads / LPH) + threadIdx.x / LPH;   // whole groups of LPH lanes
  const uint32_t n = p.tokens, each = n * (groups + 2u * heads), tile = item / each;
  item -= tile * each;
  const bool is_q = item < n * groups, is_k = !is_q && item < n * (groups + heads);
  if (!is_q) item -= n * (is_k ? groups : groups + heads);
  const int64_t t = (int64_t)tile * n + item / (is_q ? groups : heads);
  const int h = (int)(item % (is_q ? groups : heads));
  if (t >= a.T) return;
  // lanes below rot / 16 hold rotated pairs, the others the rest; e, e + half
  const int nrot = a.rot / 16;
  const bool rotated = sub < nrot, active = sub < kLanes;
  const int half = rotated ? a.rot / 2 : (D - a.rot) / 2;
  const int e = active ? (rotated ? sub * 8 : a.rot + (sub - nrot) * 8) : 0;
  RopeTables z;
  if (is_q) {
    const int h0 = h * QH;
    const uint16_t* src = a.q + t * a.q_ts + h0 * a.q_hs + e;
    u32x4 rx[QH], ry[QH];
#pragma unroll
    for (int j = 0; j < QH; ++j) {
      // (past the last head: that once more)
      const uint16_t* from = src + min(j, a.q_heads - 1 - h0) * a.q_hs;
      rx[j] = *(const u32x4*)from;
      ry[j] = *(const u32x4*)(from + half);
    }
    load_tables<INTERLEAVED>(a, a.q_weight, t, e, half, rotated, &z);
    uint16_t* dst = a.q_out + t * a.qo_ts + h0 * a.qo_hs + e;
#pragma unroll
    for (int j = 0; j < QH; ++j) {
      float x[8], y[8];
      unpack8(active ? rx[j] : u32x4{0u, 0u, 0u, 0u}, x);
      unpack8(active ? ry[j] : u32x4{0u, 0u, 0u, 0u}, y);
      norm_rotate<D, LPH, INTERLEAVED>(z, a.q_weight != nullptr, a.eps, rotated, x, y);
      if (active && h0 + j < a.q_heads) {
        store8<FAR>(dst + j * a.qo_hs, pack8(x));
        store8<FAR>(dst + j * a.qo_hs + half, pack8(y));
      }
    }
    return;
  }
  const int64_t slot = a.slots[t];
  const bool cached = slot >= 0 && slot < a.num_slots;
  const int64_t page = slot >> p.page_shift, row = slot - (page << p.page_shift), head = page * a.kv_heads + h;
  if (!is_k) {
    if (!cached) return;
    const uint16_t* src = a.v + t * a.v_ts + h * a.v_hs;
    for (int i = sub * 8; i < a.v_dim; i += LPH * 8) {              // (a block's two lanes go on together)
      float x[8];
      unpack8(*(const u32x4*)(src + i), x);
      uint32_t s;
      const uint32_t w = fp4_block(x, p.v_inv, &s);
      *(uint32_t*)(p.v_codes + ((head << p.page_shift) + row) * (a.v_dim / 2) + i / 2) = w;
      if ((sub & 1) == 0) p.v_scales[((head * (a.v_dim / 16) + i / 16) << p.page_shift) + row] = (uint8_t)s;
    }
    return;
  }
  if (!cached && !a.k_out) return;
  const uint16_t* src = a.k + t * a.k_ts + h * a.k_hs + e;
  const u32x4 rx = *(const u32x4*)src, ry = *(const u32x4*)(src + half);
  load_tables<INTERLEAVED>(a, a.k_weight, t, e, half, rotated, &z);
  float x[8], y[8];
  double xd[8], yd[8];
  unpack8(active ? rx : u32x4{0u, 0u, 0u, 0u}, x);
  unpack8(active ? ry : u32x4{0u, 0u, 0u, 0u}, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    xd[i] = x[i];
    yd[i] = y[i];
  }
  norm_rotate<D, LPH, INTERLEAVED>(z, a.k_weight != nullptr, a.eps, rotated, xd, yd);
  uint32_t s0, s1;
  const uint32_t w0 = fp4_block(xd, p.k_inv, &s0), w1 = fp4_block(yd, p.k_inv, &s1);
  if (!active) return;
  if (a.k_out) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = (float)xd[i];
      y[i] = (float)yd[i];
    }
    uint16_t* dst = a.k_out + t * a.ko_ts + h * a.ko_hs + e;
    store8<FAR>(dst, pack8(x));
    store8<FAR>(dst + half, pack8(y));
  }
  if (!cached) return;
  const int64_t at = (head << p.page_shift) + row;
  *(uint32_t*)(p.k_codes + at * (D / 2) + e / 2) = w0;
  *(uint32_t*)(p.k_codes + at * (D / 2) + (e + half) / 2) = w1;
  if ((sub & 1) == 0) {
    p.k_scales[at * (D / 16) + e / 16] = (uint8_t)s0;
    p.k_scales[at * (D / 16) + (e + half) / 16] = (uint8_t)s1;
  }
}

static int lanes_per_item(int head_dim) { return head_dim == 64 ? 4 : (head_dim == 128 ? 8 : 16); }
// As few tokens together as make whole waves of items of one kind: a wave whose lanes are of
// all three takes their times one after the other (64 tokens x 16/2 x 64: 9 us a token at a
// time, 4 us eight).  No more than that: the rows of a token lie together (8191 x 64/4 x 192:
// 92 us one at a time, 99 us four or sixteen).
static int64_t rope_fp4_tokens(int64_t groups, int64_t heads, int lanes) {
  int64_t n = 1;
  while (n * groups * lanes % 64 != 0 || n * heads * lanes % 64 != 0) n *= 2;   // (up to 64 / lanes)
  return n;
}
static int64_t rope_fp4_items(int64_t T, const moe_rope_params& p) {
  const int64_t groups = (p.q_heads + QH - 1) / QH, heads = p.kv_heads, n = rope_fp4_tokens(groups, heads, lanes_per_item(p.head_dim));
  return (T + n - 1) / n * n * (groups + 2 * heads);
}
// (a last workgroup's idle threads among them)
int64_t qk_norm_rope_fp4_threads(int64_t T, const moe_rope_params& p) {
  return rope_fp4_items(T, p) * lanes_per_item(p.head_dim) + kRopeThreads;
}

template <int D, bool INTERLEAVED, bool FAR>
static void launch_items(const RopeFp4Args& p, int64_t items, hipStream_t stream) {
  const int64_t per = kRopeThreads / lanes_per_item(D);
  hipLaunchKernelGGL((qk_norm_rope_fp4_kernel<D, INTERLEAVED, FAR>), dim3((uint32_t)((items + per - 1) / per)),
                     dim3(kRopeThreads), 0, stream, p);
}

template <int D>
static void launch_rope_fp4(const RopeFp4Args& p, int64_t items, bool interleaved, hipStream_t stream) {
  // (outputs larger than half of the 256 MB cache before HBM: see qk_norm_rope.hip)
  const bool far = p.r.T * p.r.q_heads * D * 2 > ((int64_t)128 << 20);
  if (interleaved) far ? launch_items<D, true, true>(p, items, stream) : launch_items<D, true, false>(p, items, stream);
  else far ? launch_items<D, false, true>(p, items, stream) : launch_items<D, false, false>(p, items, stream);
}

moe_status launch_qk_norm_rope_fp4(const moe_heads& q, const moe_heads& k, const moe_heads& v, int64_t T,
                                   const moe_rope_params& p, const int32_t* positions, const float* cos_sin,
                                   const float* q_weight, const float* k_weight, const moe_heads& q_out,
                                   const moe_heads* k_out, const moe_kv_cache_fp4& cache, const int32_t* slots,
                                   hipStream_t stream) {
  RopeFp4Args a;
  a.r = rope_args(q, k, &v, T, p, positions, cos_sin, q_weight, k_weight, q_out, k_out, slots);
  a.r.num_slots = cache.num_pages * cache.page_size;
  a.k_codes = (uint8_t*)cache.k;
  a.k_scales = (uint8_t*)cache.k_scale;
  a.v_codes = (uint8_t*)cache.v;
  a.v_scales = (uint8_t*)cache.v_scale;
  a.page_shift = __builtin_ctz((unsigned)cache.page_size);
  a.tokens = (uint32_t)rope_fp4_tokens((p.q_heads + QH - 1) / QH, p.kv_heads, lanes_per_item(p.head_dim));
  const int64_t items = rope_fp4_items(T, p);
  a.k_inv = 1.0f / cache.k_global;
  a.v_inv = 1.0f / cache.v_global;
  if (p.head_dim == 64) launch_rope_fp4<64>(a, items, p.interleaved, stream);
  else if (p.head_dim == 128) launch_rope_fp4<128>(a, items, p.interleaved, stream);
  else launch_rope_fp4<192>(a, items, p.interleaved, stream);
  return launch_status("moe_qk_norm_rope_fp4");
}

}  // namespace moe
