// What the decode attention calls share: the turns that a CU's workgroups take, and the
// second launch, which joins the parts that the first left of each
// output row -- unnormalised sums, maxima (base 2) and weight sums -- joined:
//   M = max m_i,  out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
#pragma once
#include "attn_common.h"

namespace moe {

constexpr int kDecSlots = 512;                      // two workgroups on each of 256 CUs

// Where the waves of a CU's two workgroups could both go on, the older's would go
// first and its workgroup end 20% before the other, which then runs alone.  So
// they take turns by tiles, two to the younger's one (blocks are handed out in
// order: the second half are the younger ones); and a narrow workgroup's few
// instructions, which keep its reads going, come before a wide one's.  64 requests
// behind 8192 tokens 78.5 -> 71.2 us (turns alone 75.0, the wide ones first 78.1),
// 96 behind 32768 150 -> 145 us, one with 131072 tokens 98 -> 95 us.
template <int LOW>
__device__ __forceinline__ void take_turns(int t) {
  const bool younger = blockIdx.x >= kDecSlots / 2;
  if ((t % 3 != 0) == younger) __builtin_amdgcn_s_setprio(LOW + 1);
  else __builtin_amdgcn_s_setprio(LOW);
}

struct JoinArgs {
  uint16_t* out;
  int64_t o_ts, o_hs;
  float* lse;
  // Prefix: part x of row b * q_heads + h is entry x * num_requests * q_heads + row.  Own
  // keys: part i of run w's share of request b is entry own + (((head * blocks_s + block) *
  // (runs + num_requests) + w + b) * run_parts + i) * rows_s + row.
  const float* part_o;                              // [entries][DV]
  const float2* part_ml;                            // [entries]: maximum (base 2), weight sum
  const int32_t* first;                             // [num_requests + 1]: tiles of the requests before
  int64_t own;
  int32_t num_requests, q_heads, kv_heads;
  int32_t prefix_parts, run_parts, runs, blocks_s, rows_s;
  float v_scale;                                    // of the values, a power of two
};

// The parts of an output row joined: WPR waves per row take every WPR-th part.
// Each wave first finds its parts' maximum (64 parts at a time, one per lane), so
// the sums' loads follow without waiting for one another.
template <int DV, int WPR>
__global__ __launch_bounds__(WPR <= 4 ? 256 : WPR * 64) void attn_join_kernel(JoinArgs a) {
  constexpr int kWaves = WPR <= 4 ? 4 : WPR, kRows = kWaves / WPR;
  __shared__ float2 red[kWaves][64];
  __shared__ float2 ml[kWaves];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = wv % WPR;
  const int Hall = a.num_requests * a.q_heads;
  const int at_row = blockIdx.x * kRows + wv / WPR;
  const bool live = at_row < Hall;                                  // whole waves; a row's waves agree
  const int b = min(at_row, Hall - 1) / a.q_heads, hq = min(at_row, Hall - 1) % a.q_heads;
  constexpr int E = DV / 64;                                        // values per lane
  float M = neg_inf(), L = 0.0f, o[2] = {0.0f, 0.0f};
  if (live) {
    // own parts: run_parts for each run that the request's tiles lie in
    const int np = a.prefix_parts;
    int n = np, run0 = 0;
    if (a.runs > 0) {
      const int t0 = a.first[b], t1 = a.first[b + 1], each = (a.first[a.num_requests] + a.runs - 1) / a.runs;
      if (t1 > t0) {
        run0 = t0 / each;
        n += a.run_parts * ((t1 - 1) / each - run0 + 1);
      }
    }
    const int G = a.q_heads / a.kv_heads, kvh = hq / G, g = hq % G, block = g / a.rows_s;
    const int64_t own = a.own + ((int64_t)(kvh * a.blocks_s + block) * (a.runs + a.num_requests) + run0 + b) * a.run_parts * a.rows_s +
                        g - block * a.rows_s;
    auto entry = [&](int x) { return x < np ? (int64_t)x * Hall + at_row : own + (int64_t)(x - np) * a.rows_s; };
    const int mine = (n - sub + WPR - 1) / WPR;                     // parts sub, sub + WPR, ...
    for (int base = 0; base < mine; base += 64) {
      const int cnt = min(64, mine - base);
      float2 x = float2{neg_inf(), 0.0f};
      if (lane < cnt) x = a.part_ml[entry(sub + (base + lane) * WPR)];
      float y[8][2];
      auto load = [&](int q0) {                                     // 8 under way; the first with the maxima
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float* src = a.part_o + entry(sub + (base + min(q0 + u, cnt - 1)) * WPR) * DV + lane * E;
          y[u][0] = src[0];
          if (E == 2) y[u][1] = src[1];
        }
      };
      load(0);
      float mx = x.x;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
      const float M1 = fmaxf(M, mx), ref = M1 == neg_inf() ? 0.0f : M1;
      const float e = __builtin_amdgcn_exp2f(x.x - ref), e0 = __builtin_amdgcn_exp2f(M - ref);
      float l = x.y * e;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) l += __shfl_xor(l, d);
      L = L * e0 + l;
      M = M1;
#pragma unroll
      for (int j = 0; j < E; ++j) o[j] *= e0;
      for (int q0 = 0; q0 < cnt; q0 += 8) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (q0 + u >= cnt) break;
          const float ep = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e), q0 + u));
          o[0] = fmaf(ep, y[u][0], o[0]);
          if (E == 2) o[1] = fmaf(ep, y[u][1], o[1]);
        }
        if (q0 + 8 < cnt) load(q0 + 8);
      }
    }
  }
  if (WPR > 1) {
    red[wv][lane] = float2{o[0], o[1]};
    if (lane == 0) ml[wv] = float2{M, L};
    __syncthreads();
    if (sub != 0) return;
    float M1 = M;
#pragma unroll
    for (int i = 1; i < WPR; ++i) M1 = fmaxf(M1, ml[wv + i].x);
    const float ref = M1 == neg_inf() ? 0.0f : M1;
    float e = __builtin_amdgcn_exp2f(M - ref);
    L *= e;
    o[0] *= e;
    o[1] *= e;
#pragma unroll
    for (int i = 1; i < WPR; ++i) {
      e = __builtin_amdgcn_exp2f(ml[wv + i].x - ref);
      const float2 y = red[wv + i][lane];
      L = fmaf(e, ml[wv + i].y, L);
      o[0] = fmaf(e, y.x, o[0]);
      o[1] = fmaf(e, y.y, o[1]);
    }
    M = M1;
  }
  if (!live) return;
  const float inv = L == 0.0f ? 0.0f : a.v_scale / L;
  uint16_t* dst = a.out + b * a.o_ts + hq * a.o_hs + lane * E;
  if (E == 2) *(uint32_t*)dst = cvt_bf16x2(o[0] * inv, o[1] * inv);
  else *dst = (uint16_t)f32_to_bf16_bits(o[0] * inv);
  if (a.lse && lane == 0) a.lse[at_row] = L == 0.0f ? neg_inf() : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// Waves per row: as many as leave each 8 parts or so, one round of loads (a request's own
// parts: run_parts per run it lies in, on average runs / requests of them).
inline int join_waves(int prefix_parts, int run_parts, int runs, int num_requests) {
  const int parts = prefix_parts + run_parts * (1 + runs / num_requests);
  return parts <= 16 ? 1 : (parts <= 48 ? 4 : 16);
}

template <int DV>
static void launch_join(const JoinArgs& a, hipStream_t stream) {
  const uint32_t rows = (uint32_t)(a.num_requests * a.q_heads);
  const int waves = join_waves(a.prefix_parts, a.run_parts, a.runs, a.num_requests);
  if (waves == 1) hipLaunchKernelGGL((attn_join_kernel<DV, 1>), dim3((rows + 3) / 4), dim3(256), 0, stream, a);
  else if (waves == 4) hipLaunchKernelGGL((attn_join_kernel<DV, 4>), dim3(rows), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((attn_join_kernel<DV, 16>), dim3(rows), dim3(1024), 0, stream, a);
}

}  // namespace moe
