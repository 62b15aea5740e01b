// The residual stream between two blocks in one pass over its rows:
//   b = x * rsqrt(mean(x^2) + eps) * post_weight    (norm behind the block; none: b = x)
//   h = residual + scale * gate * b                 (gate of each channel or each value)
//   y = h * rsqrt(mean(h^2) + eps) * weight         (norm before the next block)
// in float, h and y each rounded once to bf16 (y comes from the unrounded h).
//
// Memory traffic is all there is: a workgroup per row keeps the row in registers, so
// x, residual and gate are read once and h and y written once.  8191 x 4096 with both norms and a
// channel gate (268 MB): 54 us, 5.0 TB/s where a large copy reaches 5.1; non-temporal loads or
// stores are within 5% of that, rows dealt to the XCDs in blocks 12% slower.  64 x 4096: 3.3 us, a
// launch's latency.
#include <algorithm>

#include "common.h"

namespace moe {

struct BlockNormArgs {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* gate;                             // of each value
  const float* channel_gate;
  const float* post_weight;
  const float* weight;
  uint16_t* h;
  uint16_t* y;
  int64_t x_ts, r_ts, g_ts, h_ts, y_ts;
  int32_t hidden;
  float scale, eps, inv;                            // inv: 1 / hidden
};

// Sum over the workgroup (every thread gets it, in the same order whatever the row).
template <int WAVES>
__device__ __forceinline__ float row_sum(float x, float* part) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  if (WAVES == 1) return x;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) sum += part[w];
  return sum;
}

__device__ __forceinline__ void load_row8(const uint16_t* p, float (&x)[8]) {
  const u32x4 w = *(const u32x4*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void load_f32x8(const float* p, float (&x)[8]) {
  const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = a[i];
    x[4 + i] = b[i];
  }
}
__device__ __forceinline__ u32x4 pack_row8(const float (&x)[8]) {
  return u32x4{cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]), cvt_bf16x2(x[6], x[7])};
}

// WAVES waves per row, N pieces of 8 values per thread.
template <int WAVES, int N>
__global__ __launch_bounds__(WAVES * 64) void block_norm_kernel(BlockNormArgs a) {
  __shared__ float part[2][WAVES];
  const int64_t t = blockIdx.x;
  const uint16_t* x = a.x + t * a.x_ts;
  float b[N][8];
  const int e0 = threadIdx.x * 8;
  constexpr int kStep = WAVES * 64 * 8;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i * kStep;
    if (e < a.hidden) load_row8(x + e, b[i]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) b[i][j] = 0.0f;
  }
  float r[N][8];
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e0 + i * kStep < a.hidden) load_row8(a.residual + t * a.r_ts + e0 + i * kStep, r[i]);
  }
  if (a.post_weight) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(b[i][j], b[i][j], ss);
    const float k = 1.0f / sqrtf(row_sum<WAVES>(ss, part[0]) * a.inv + a.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (e0 + i * kStep >= a.hidden) continue;
      float w[8];
      load_f32x8(a.post_weight + e0 + i * kStep, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) b[i][j] = b[i][j] * k * w[j];
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i * kStep;
    if (e >= a.hidden) continue;
    if (a.gate || a.channel_gate) {
      float g[8];
      if (a.gate) load_row8(a.gate + t * a.g_ts + e, g);
      else load_f32x8(a.channel_gate + e, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) b[i][j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      b[i][j] = a.residual ? fmaf(a.scale, b[i][j], r[i][j]) : a.scale * b[i][j];
      ss = fmaf(b[i][j], b[i][j], ss);
    }
    if (a.h) *(u32x4*)(a.h + t * a.h_ts + e) = pack_row8(b[i]);
  }
  if (!a.y) return;
  const float k = 1.0f / sqrtf(row_sum<WAVES>(ss, part[1]) * a.inv + a.eps);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = e0 + i * kStep;
    if (e >= a.hidden) continue;
    float w[8];
    load_f32x8(a.weight + e, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) b[i][j] = b[i][j] * k * w[j];
    *(u32x4*)(a.y + t * a.y_ts + e) = pack_row8(b[i]);
  }
}

int block_norm_max_hidden() { return 32768; }

// (2^21 rows at a time: a launch's threads are counted in 32 bits)
template <int WAVES, int N>
static void launch_norm(BlockNormArgs a, int64_t T, hipStream_t stream) {
  const int64_t most = (int64_t)1 << 21;
  for (; T > 0; T -= most) {
    hipLaunchKernelGGL((block_norm_kernel<WAVES, N>), dim3((uint32_t)std::min(T, most)), dim3(WAVES * 64), 0, stream, a);
    a.x += most * a.x_ts;
    a.residual += a.residual ? most * a.r_ts : 0;
    a.gate += a.gate ? most * a.g_ts : 0;
    a.h += a.h ? most * a.h_ts : 0;
    a.y += a.y ? most * a.y_ts : 0;
  }
}

moe_status launch_block_norm(const moe_rows& x, int64_t T, int hidden, const moe_rows* residual, const float* post_weight,
                             const moe_rows* gate, const float* channel_gate, float scale, const float* weight, float eps,
                             const moe_rows* h, const moe_rows* y, hipStream_t stream) {
  BlockNormArgs a = {};
  a.x = (const uint16_t*)x.data;
  a.x_ts = x.stride;
  a.residual = residual ? (const uint16_t*)residual->data : nullptr;
  a.r_ts = residual ? residual->stride : 0;
  a.gate = gate ? (const uint16_t*)gate->data : nullptr;
  a.g_ts = gate ? gate->stride : 0;
  a.channel_gate = channel_gate;
  a.post_weight = post_weight;
  a.weight = weight;
  a.h = h ? (uint16_t*)h->data : nullptr;
  a.h_ts = h ? h->stride : 0;
  a.y = y ? (uint16_t*)y->data : nullptr;
  a.y_ts = y ? y->stride : 0;
  a.hidden = hidden;
  a.scale = scale;
  a.eps = eps;
  a.inv = 1.0f / (float)hidden;
  // as many waves as leave each thread one piece, if there are so many (8 for 4 with two pieces:
  // 8191 x 4096 55.6 -> 53.8 us, 64 x 4096 4.3 -> 3.3; 16 for 4 with four: 4000 x 8192 59 -> 53; 2 for 4
  // that are half empty: 20000 x 1024 42.6 -> 32.6)
  if (hidden <= 512) launch_norm<1, 1>(a, T, stream);
  else if (hidden <= 1024) launch_norm<2, 1>(a, T, stream);
  else if (hidden <= 2048) launch_norm<4, 1>(a, T, stream);
  else if (hidden <= 4096) launch_norm<8, 1>(a, T, stream);
  else if (hidden <= 8192) launch_norm<16, 1>(a, T, stream);
  else if (hidden <= 16384) launch_norm<16, 2>(a, T, stream);
  else launch_norm<16, 4>(a, T, stream);
  return launch_status("moe_block_norm");
}

}  // namespace moe
